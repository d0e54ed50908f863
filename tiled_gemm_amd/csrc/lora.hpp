// Low-rank adapters beside a shared projection: the second half, inside the
// projection's kernel (the first half, v / s = x down^T, is lora.hip).
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
// v goes to the matrix unit as a sum of bf16 numbers, for as many MFMAs of a
// product that is 1 to 3% of the projection's: of two (within 2^-16) where the
// output is bf16, as rounding v to one would add an error as large as the
// output's own rounding where the adapters' share of z is large; of three (within
// 2^-24) where it is fp32 or an fp32 partial tile.  v comes as fp32 partial sums over parts of
// K, which the reader adds.
#pragma once

#include "device.hpp"

namespace tg {

// bf16 numbers that stand for one of v.
template <int OUT>
constexpr int lora_planes() { return OUT == kOutF32 ? 3 : 2; }

// Eight fp32 numbers as the sums of P bf16 operands: each but the last cuts the
// number off after 8 bits, so what is left has the number's sign, and where
// nothing is left 2^-28 of the number follows, which no fp32 sum beside the number
// holds.  So the operands are infinite, NaN, zero or of one sign together, and
// against an infinite element of `up` their products are one infinity (while |v| is
// above 2^-105, where 2^-28 of it is still a number).  Rounded to nearest instead, the
// remainder of an infinity is NaN, and any other may have the other sign or be zero:
// NaN for an infinite z.  (No slower, either: 150 / 150 us in packed prompts; a check
// of every product for infinities took 160.)
template <int P>
__device__ inline void split_bf16(const f32x4 &a, const f32x4 &b, u32x4 (&o)[P])
{
    float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int p = 0; p < P - 1; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = __builtin_bit_cast(uint32_t, v[2 * i]), hi = __builtin_bit_cast(uint32_t, v[2 * i + 1]);
            o[p][i] = lo >> 16 | (hi & 0xFFFF0000u);
            v[2 * i] = lo & 0xFFFF ? v[2 * i] - bf16_lo(o[p][i]) : v[2 * i] * 0x1p-28f;
            v[2 * i + 1] = hi & 0xFFFF ? v[2 * i + 1] - bf16_hi(o[p][i]) : v[2 * i + 1] * 0x1p-28f;
        }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[P - 1][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
}

// This lane's place among the columns of `up`: its row r16 of each column block
// and the 8 ranks from r0 + 8 q, as byte offsets (past the matrix for columns
// past N and ranks past the last).
template <int FN>
struct LoraCols {
    uint32_t off[FN];
    uint32_t bytes;              // of one adapter's matrix
    __device__ LoraCols(const LoraArgs &lo, int N, int col0, int r0)
    {
        const int l = lane_id(), r = r0 + 8 * (l >> 4);
        const uint32_t pitch = (uint32_t)lo.rank * 2u;
        bytes = (uint32_t)N * pitch;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int col = col0 + j * 16 + (l & 15);
            off[j] = keep_or_oob(col < N && r < lo.rank, (uint32_t)col * pitch + (uint32_t)r * 2u);
        }
    }
    __device__ void load(const LoraArgs &lo, int e, u32x4 (&b)[FN]) const
    {
        // (one adapter for the whole wave, which the compiler cannot see)
        const auto ru = make_rsrc((const uint8_t *)lo.up + (size_t)__builtin_amdgcn_readfirstlane(e) * bytes, bytes);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            b[j] = buf_load16(ru, off[j], 0);
    }
};

// acc += v b^T for the rows whose bit is set in `same` (bit 16 i + r: row r of
// block i), 32 ranks.
template <int P, int CH, int FN>
__device__ inline void lora_add(f32x4 (*acc)[FN], const u32x4 (&v)[CH][P], const u32x4 (&b)[FN], unsigned long long same)
{
    const int r16 = lane_id() & 15;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        if (((same >> (i * 16)) & 0xFFFF) == 0)      // none of this block's rows (the same in every lane)
            continue;
        const bool mine = (same >> (i * 16 + r16)) & 1;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < P; ++p)
                t = mfma_bf16(b[j], v[i][p], t);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[i][j][c] += mine ? t[c] : 0.f;
        }
    }
}

// The adapter of one row per lane (-1: none).
__device__ inline int lora_id(const LoraArgs &lo, bool there, int row)
{
    const int id = there ? lo.adapter[row] : -1;
    return (uint32_t)id < (uint32_t)lo.adapters ? id : -1;
}

// The factor of a row with the adapter `id` (any, where it has none: its v is not used).
__device__ inline float lora_scale(const LoraArgs &lo, int id)
{
    return lo.scale ? lo.scale[(uint32_t)id < (uint32_t)lo.adapters ? id : 0] : 1.f;
}

// Eight ranks of a row of v from column c on: its parts added, in their order, and
// scaled.  (The parts one by one would make NaN of an infinite scale where they
// differ in sign or are zero, and of a large one whose products with them
// overflow.  Reading the scale here costs 32 decode rows 0.8 of 36 us, tiles nothing
// that shows.)
// (Ranks past the last, up to a multiple of 32, are zeros to the matrix unit; they
// are neither stored nor read: an infinite x times the zeros that its rows of
// `down` would be is NaN.)
__device__ inline void lora_v8(const LoraArgs &lo, size_t row, int c, float scale, f32x4 &a, f32x4 &b)
{
    const float *const p = (const float *)lo.v + row * lo.rank_pad + c;
    const size_t part = (size_t)lo.M * lo.rank_pad;
    f32x4 x[kLoraParts], y[kLoraParts];
#pragma unroll
    for (int s = 0; s < kLoraParts; ++s) {
        const float *const at = p + (s < lo.parts ? s : 0) * part;      // in flight together
        x[s] = *(const f32x4 *)at;
        y[s] = *(const f32x4 *)(at + 4);
    }
    a = x[0];
    b = y[0];
#pragma unroll
    for (int s = 1; s < kLoraParts; ++s) {
        if (s < lo.parts) {
            a += x[s];
            b += y[s];
        }
    }
    a *= scale;
    b *= scale;
}

// LDS of lora_tail: 32 ranks of the tile's rows, P times.
template <int BM, int P>
constexpr int lora_lds_bytes() { return BM * 64 * P; }

// acc[i][j] of a tile wave: row block i holds the tile's rows row0 + 16 i .., of
// which `rows` exist, from row m0 of C on.  All waves of the tile's workgroup
// call it: v goes through LDS, so that it is read, added up and split once per
// tile and not once per wave (with the parts of K that are added up here:
// 8192 x 8192 x 2048, rank 32, 337 -> 328 us).  LDS may still be read by other waves
// before the call and after it.  What it costs with one adapter is hard to see
// (that shape's kernel: 287 us, 286 without adapters; 2000 x 4096 x 4160, rank 64: 103
// and 98); each adapter beyond the first among a wave's 64 rows takes some 250
// cycles, a chain of ballots and dependent MFMAs.  Their columns, loaded three
// adapters ahead, are not waited for (five or six ahead change nothing).
template <int BM, int THREADS, int P, int FM, int FN>
__device__ inline void lora_tail(const LoraArgs &lo, f32x4 (&acc)[FM][FN], uint8_t *lds, int m0, int rows, int row0,
                                 int col0, int N)
{
    // Row blocks at a time: a row per lane, and what the registers hold.
    constexpr int MOST = P == 2 ? 4 : 2, CH = FM < MOST ? FM : MOST;
    constexpr int CHUNKS = FM / CH;
    static_assert(FM % CH == 0, "whole chunks");
    const int l = lane_id(), q = l >> 4, r16 = l & 15;
    int id[CHUNKS];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const int row = row0 + 16 * CH * c + l;
        id[c] = lora_id(lo, l < 16 * CH && row < rows, m0 + row);
    }
    constexpr int ITEMS = BM * 4 / THREADS;
    static_assert(BM * 4 % THREADS == 0, "as many pieces of v for every thread");
    float scale[ITEMS];
#pragma unroll
    for (int u = 0; u < ITEMS; ++u) {
        const int row = (threadIdx.x + u * THREADS) >> 2;
        scale[u] = lora_scale(lo, lo.adapter[m0 + min(row, rows - 1)]);
    }
    for (int r0 = 0; r0 < lo.rank_pad; r0 += 32) {
        const LoraCols<FN> cols(lo, N, col0, r0);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            const int it = threadIdx.x + u * THREADS, row = it >> 2, c = it & 3;
            f32x4 va = {0.f, 0.f, 0.f, 0.f}, vb = va;
            if (row < rows && r0 + 8 * c < lo.rank)
                lora_v8(lo, (size_t)(m0 + row), r0 + 8 * c, scale[u], va, vb);
            u32x4 o[P];
            split_bf16<P>(va, vb, o);
#pragma unroll
            for (int p = 0; p < P; ++p)
                *(u32x4 *)(lds + p * BM * 64 + it * 16) = o[p];
        }
        __syncthreads();
        u32x4 b[3][FN];
        int have = -1;                               // the adapter whose columns b[0] holds
        static_for<CHUNKS>([&](auto c_c) {
            constexpr int C = decltype(c_c)::value;
            unsigned long long left = __ballot(id[C] >= 0);
            if (!left)
                return;
            auto pop = [&]() {                       // the next adapter among the chunk's rows, or -1
                if (!left)
                    return -1;
                const int e = __builtin_amdgcn_readlane(id[C], __builtin_ctzll(left));
                left &= ~__ballot(id[C] == e);
                return e;
            };
            int e0 = pop(), e1 = pop();
            if (e0 != have)
                cols.load(lo, e0, b[0]);
            if (e1 >= 0)
                cols.load(lo, e1, b[1]);
            u32x4 v[CH][P];
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    v[i][p] = lds_load16(lds + p * BM * 64 + (row0 + 16 * (C * CH + i) + r16) * 64 + q * 16);
            // One adapter's products from `now` while the columns of the one after
            // the next start on their way to `ahead` (a decode row's adapter has
            // not been read before: its columns come from HBM); false after the last.
            auto one = [&](const u32x4 (&now)[FN], u32x4 (&ahead)[FN]) {
                const unsigned long long same = __ballot(id[C] == e0);
                have = e0;
                e0 = e1;
                e1 = pop();
                if (e1 >= 0)
                    cols.load(lo, e1, ahead);
                lora_add<P, CH, FN>(&acc[C * CH], v, now, same);
                return e0 >= 0;
            };
            while (one(b[0], b[2])) {
                have = -1;
                if (!one(b[1], b[0]) || !one(b[2], b[1])) {
                    have = -1;
                    break;
                }
            }
        });
    }
    __syncthreads();
}

// The same for a few rows (M <= 64), the adapters shared out to `waves` waves:
// wave w of them takes every waves-th that occurs.  acc: sums to be added to the
// other waves'.
template <int P, int MB, int FN>
__device__ inline void lora_skinny(const LoraArgs &lo, f32x4 (&acc)[MB][FN], int M, int N, int col0, int w, int waves)
{
    const int l = lane_id(), q = l >> 4, r16 = l & 15;
    const int id = lora_id(lo, l < M, l);
    float scale[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
        scale[i] = lora_scale(lo, lo.adapter[min(16 * i + r16, M - 1)]);
    // The wave's next adapter: its first row's, every waves-th of those left.
    unsigned long long left = 0;
    int n = 0;
    auto next = [&](unsigned long long *same) {
        while (left) {
            const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
            *same = __ballot(id == e);
            left &= ~*same;
            if (n++ % waves == w)
                return e;
        }
        return -1;
    };
    for (int r0 = 0; r0 < lo.rank_pad; r0 += 32) {
        const LoraCols<FN> cols(lo, N, col0, r0);
        left = __ballot(id >= 0);
        n = 0;
        unsigned long long same = 0, same1 = 0;
        int e = next(&same);
        if (e < 0)
            return;                                  // fewer adapters than waves
        u32x4 b[FN], b1[FN];
        cols.load(lo, e, b);
        u32x4 v[MB][P];
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            f32x4 va = {0.f, 0.f, 0.f, 0.f}, vb = va;
            if (16 * i + r16 < M && r0 + 8 * q < lo.rank)
                lora_v8(lo, 16 * i + r16, r0 + 8 * q, scale[i], va, vb);
            split_bf16<P>(va, vb, v[i]);
        }
        while (e >= 0) {
            const int e1 = next(&same1);
            if (e1 >= 0)
                cols.load(lo, e1, b1);               // in flight while this one's products run
            lora_add<P, MB, FN>(acc, v, b, same);
            e = e1;
            same = same1;
#pragma unroll
            for (int j = 0; j < FN; ++j)
                b[j] = b1[j];
        }
    }
}

}  // namespace tg
