// Low-rank adapters beside a shared projection: the second half, inside the
// projection's kernel (the first half, v = s x down^T, is lora.hip).
//
//   z[m][n] = sum_k x[m][k] b[n][k] + sum_r v[m][r] up_a[n][r],     a the adapter of row m
//
// The sum over r is a few more MFMAs on the accumulators that the main loop
// leaves, before the epilogue, so z is never written on the way.  Rows of
// several adapters share a block of 16: the product is made once per adapter
// that occurs among a wave's rows and each row takes the one of its own.
// (Choosing the finished sums rather than clearing the other rows' v keeps an
// infinity or NaN of one adapter's matrices out of the other adapters' rows.)
//
// v comes as fp32 (in `parts` partial sums over K) and goes to the matrix unit
// as two bf16 numbers, v = hi + lo within 2^-17 of it, for twice the MFMAs of a
// product that is 1 to 3% of the projection's: rounding v to one bf16 would add
// an error as large as the output's own rounding where the adapters' share of z
// is large.
#pragma once

#include "device.hpp"

namespace tg {

// Eight fp32 numbers as bf16 operands hi + lo.
__device__ inline void split_bf16(const f32x4 &a, const f32x4 &b, u32x4 &hi, u32x4 &lo)
{
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        hi[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        lo[i] = pack_bf16x2(v[2 * i] - bf16_lo(hi[i]), v[2 * i + 1] - bf16_hi(hi[i]));
    }
}

// acc += v up_e^T for the rows whose bit is set in `same` (bit 16 i + r: row r of
// block i).  row[i]: this lane's row of block i within the tile; col0: the wave's
// first column.
template <int CH, int FN>
__device__ inline void lora_add(const LoraArgs &lo, int m0, int rows, int N, f32x4 (*acc)[FN], const int (&row)[CH],
                                unsigned long long same, int e, int col0)
{
    const int l = lane_id(), q = l >> 4, r16 = l & 15;
    const uint32_t pitch = (uint32_t)lo.rank_pad * 4u, upitch = (uint32_t)lo.rank * 2u;
    const auto ru = make_rsrc((const uint8_t *)lo.up + (size_t)e * (size_t)N * upitch, (uint32_t)N * upitch);
    f32x4 t[CH][FN];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            t[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int r0 = 0; r0 < lo.rank_pad; r0 += 32) {
        u32x4 b[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int col = col0 + j * 16 + r16;
            b[j] = buf_load16(ru, keep_or_oob(col < N && r0 + 8 * q < lo.rank,
                                              (uint32_t)col * upitch + (uint32_t)(r0 + 8 * q) * 2u), 0);
        }
        f32x4 va[CH], vb[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i)
            va[i] = vb[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < lo.parts; ++s) {
            const auto rv = make_rsrc(lo.v + ((size_t)s * lo.M + m0) * lo.rank_pad, (uint32_t)rows * pitch);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const uint32_t off = keep_or_oob(row[i] < rows, (uint32_t)row[i] * pitch + (uint32_t)(r0 + 8 * q) * 4u);
                va[i] += __builtin_bit_cast(f32x4, buf_load16(rv, off, 0));
                vb[i] += __builtin_bit_cast(f32x4, buf_load16(rv, off, 16));
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            u32x4 hi, low;
            split_bf16(va[i], vb[i], hi, low);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                t[i][j] = mfma_bf16(b[j], hi, t[i][j]);
                t[i][j] = mfma_bf16(b[j], low, t[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const bool mine = (same >> (i * 16 + r16)) & 1;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[i][j][c] += mine ? t[i][j][c] : 0.f;
    }
}

// The adapters of a wave's CH row blocks, one row per lane (-1: none); the lane
// of row r of block i is 16 i + r.
template <int CH>
__device__ inline int lora_ids(const LoraArgs &lo, int m0, int rows, int first_row)
{
    const int l = lane_id(), row = first_row + l;
    const int id = l < 16 * CH && row < rows ? lo.adapter[m0 + row] : -1;
    return (uint32_t)id < (uint32_t)lo.adapters ? id : -1;
}

// acc[i][j] of a tile wave: row block i holds the tile's rows row0 + 16 i .., of
// which `rows` exist, from row m0 of C on.
template <int FM, int FN>
__device__ inline void lora_tail(const LoraArgs &lo, f32x4 (&acc)[FM][FN], int m0, int rows, int row0, int col0, int N)
{
    // Row blocks at a time: as many sums beside the accumulators as still
    // leave registers for the operands.
    constexpr int CH = FN >= 4 ? 2 : (FM < 4 ? FM : 4);
    static_assert(FM % CH == 0, "whole chunks");
    static_for<FM / CH>([&](auto c_c) {
        constexpr int C = decltype(c_c)::value * CH;
        const int id = lora_ids<CH>(lo, m0, rows, row0 + 16 * C);
        int row[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i)
            row[i] = row0 + 16 * (C + i) + (lane_id() & 15);
        for (unsigned long long left = __ballot(id >= 0); left;) {
            const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
            const unsigned long long same = __ballot(id == e);
            left &= ~same;
            lora_add<CH, FN>(lo, m0, rows, N, &acc[C], row, same, e, col0);
        }
    });
}

// The same for a few rows (M <= 64), the adapters shared out to `waves` waves:
// wave w of them takes every waves-th that occurs.  acc: sums to be added to the
// other waves'.
template <int MB, int FN>
__device__ inline void lora_skinny(const LoraArgs &lo, f32x4 (&acc)[MB][FN], int M, int N, int col0, int w, int waves)
{
    const int id = lora_ids<MB>(lo, 0, M, 0);
    int row[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
        row[i] = 16 * i + (lane_id() & 15);
    int n = 0;
    for (unsigned long long left = __ballot(id >= 0); left; ++n) {
        const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const unsigned long long same = __ballot(id == e);
        left &= ~same;
        if (n % waves == w)
            lora_add<MB, FN>(lo, 0, M, N, acc, row, same, e, col0);
    }
}

}  // namespace tg
