// Products of a few gathered rows with a few blocks of 16 weight rows, both read
// straight from global memory into registers in MFMA order, K split over the
// waves of a workgroup.
#pragma once

#include "device.hpp"

namespace tg {

constexpr int kStreamWaves = 8;
constexpr int kStreamThreads = 64 * kStreamWaves;

// One row of a wave's sums: 16 NB columns, padded to spread over the banks.
template <int NB>
constexpr int stream_pitch() { return 16 * NB + 1; }

// Eight e4m3 elements (two words) as an MFMA operand of eight bf16: exact.
__device__ inline u32x4 fp8x8_to_bf16(uint32_t lo, uint32_t hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
    return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                 __builtin_bit_cast(uint32_t, d)};
}

// Products of 16 MB rows with NB blocks of 16 weight rows over the 64-byte steps
// step0 .. step0 + steps - 1 of K; the waves' sums end up in red, to be added
// over the waves (stream_sum).
//   rX      the rows' array; xoff[i]: byte offset of this lane's row (l % 16 of
//           row block i), past the array for rows that are not there
//   rB[j]   weight block j: 16 rows of kb bytes (or their image)
// Lane 16 q + r holds bytes 16 q .. of row r of a step, one MFMA of bf16 or two
// of e4m3 (E8: elements 16 q .. + 7 and + 8 .. + 15).  Two sets of U steps are in
// flight per wave.  find(rB) names the weight blocks; it is called once the first
// loads of x are on their way, so that what it waits for (which adapter the rows
// have, say) is waited for beside them.
template <int MB, int NB, bool E8, bool PRE, int U, typename Find>
__device__ inline void stream_product(__amdgpu_buffer_rsrc_t rX, const uint32_t (&xoff)[MB], Find find, uint32_t kb,
                                      int step0, int steps, float (*red)[16 * MB][stream_pitch<NB>()])
{
    constexpr int H = E8 ? 2 : 1;                    // MFMAs (and 16-byte loads of a row of x) per step
    const int w = wave_id(), l = lane_id(), q = l >> 4, r16 = l & 15;
    const int first = step0 + w * steps / kStreamWaves, nt = step0 + (w + 1) * steps / kStreamWaves - first;
    const uint32_t boff = PRE ? (uint32_t)l * 16u : (uint32_t)r16 * kb + (uint32_t)q * 16u;
    struct Set {
        u32x4 b[U][NB];
        u32x4 x[U][MB][H];
    };
    __amdgpu_buffer_rsrc_t rB[NB];
    auto load_b = [&](int t0, Set &s) {
#pragma unroll
        for (int j = 0; j < NB; ++j)                 // (steps inside: the halves of a line one after the other)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = t0 + u < nt;
                const uint32_t k = in ? (uint32_t)(first + t0 + u) : 0u;
                s.b[u][j] = buf_load16(rB[j], keep_or_oob(in, boff), k * (PRE ? 1024u : 64u));
            }
    };
    auto load_x = [&](int t0, Set &s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = t0 + u < nt;
            const uint32_t k = in ? (uint32_t)(first + t0 + u) : 0u;
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int h = 0; h < H; ++h)
                    s.x[u][i][h] = buf_load16(rX, keep_or_oob(in, xoff[i] + (uint32_t)(q * 16 * H + 16 * h)),
                                              k * (64u * H));
        }
    };
    auto load = [&](int t0, Set &s) {
        load_b(t0, s);
        load_x(t0, s);
        issue_fence();
    };
    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const Set &s) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const u32x4 b = E8 ? fp8x8_to_bf16(s.b[u][j][2 * h], s.b[u][j][2 * h + (E8 ? 1 : 0)]) : s.b[u][j];
#pragma unroll
                    for (int i = 0; i < MB; ++i)
                        acc[i][j] = mfma_bf16(b, s.x[u][i][h], acc[i][j]);
                }
    };
    Set s0, s1;
    load_x(0, s0);
    issue_fence();
    find(rB);
    load_b(0, s0);
    load(U, s1);
    for (int t = 2 * U; t < nt; t += 2 * U) {
        compute(s0);
        load(t, s0);
        compute(s1);
        load(t + U, s1);
    }
    compute(s0);
    compute(s1);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                red[w][i * 16 + r16][j * 16 + 4 * q + v] = acc[i][j][v];
}

// The sum over the waves, in their order.
template <int MB, int NB>
__device__ inline float stream_sum(const float (*red)[16 * MB][stream_pitch<NB>()], int row, int col)
{
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kStreamWaves; ++w)
        s += red[w][row][col];
    return s;
}

}  // namespace tg
