// Low-rank adapters of many requests, the first half:
//
//   v[m][r] = s_a sum_k x[m][k] down_a[r][k],     a the adapter of row m
//
// for the projection's kernel to finish (lora.hpp), as fp32 or as two bf16
// numbers.  Two forms, by the number of rows:
//   * up to kLoraFewRows (decode): the adapters' matrices are the bytes, most
//     rows have one of their own, and a workgroup alone would take long over
//     one.  So a workgroup takes one adapter of 16 rows, 16 of its ranks and one
//     part of K.
//   * above (prompts, training): x is the bytes, and blocks of rows mostly have
//     one adapter.  A workgroup takes the first adapter of 16 or 32 rows with up
//     to 64 ranks at once, x read once for them.  The further adapters of a
//     group of 64 rows (decode rows in front of the prompts, a prompt's end) are
//     shared out to kLoraMore workgroups more: one after the other in the
//     block's own workgroup, 16 of them took 260 us (4001 x 4160, rank 64).
#include "stream.hpp"

namespace tg {

namespace {

constexpr int kLoraMore = 15;

// The n-th adapter (in the order of its first row) among the rows of `mask`, or
// -1; same: its rows.  id: one row per lane, -1 without an adapter.
__device__ inline int lora_nth(int id, unsigned long long mask, int n, unsigned long long *same)
{
    unsigned long long left = __ballot(id >= 0) & mask;
    while (left) {
        const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        *same = __ballot(id == e) & mask;
        if (n-- == 0)
            return e;
        left &= ~*same;
    }
    return -1;
}

// Adapter e's product with the 16 MB rows from m0 on, ranks 16 NB rb .., K steps
// of part `part`; stored for the rows of `same` (bit r: row m0 + r).
template <int MB, int NB>
__device__ inline void lora_down(const LoraArgs &a, int m0, int e, unsigned long long same, int rb, int part,
                                 float (*red)[16 * MB][stream_pitch<NB>()])
{
    const int r16 = lane_id() & 15;
    const uint32_t kb = (uint32_t)a.K * 2u;
    const int steps = (int)(kb / 64), per = (steps + a.parts - 1) / a.parts;
    const int step0 = min(part * per, steps), n_steps = min(per, steps - step0);
    const auto rX = make_rsrc((const uint8_t *)a.x + (size_t)m0 * kb, (uint32_t)min(a.M - m0, 16 * MB) * kb);
    uint32_t xoff[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
        xoff[i] = keep_or_oob(m0 + i * 16 + r16 < a.M, (uint32_t)(i * 16 + r16) * kb);
    __amdgpu_buffer_rsrc_t rB[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        // ranks past the last (of a padded block) read zeros
        const int r = (rb * NB + j) * 16;
        rB[j] = make_rsrc((const uint8_t *)a.down + ((size_t)e * a.rank + min(r, a.rank)) * kb,
                          (uint32_t)max(0, min(a.rank - r, 16)) * kb);
    }
    stream_product<MB, NB, false, false, NB == 1 ? 4 : 2>(rX, xoff, rB, kb, step0, n_steps, red);
    __syncthreads();
    const float s = a.scale ? a.scale[e] : 1.f;
    for (int o = threadIdx.x; o < 16 * MB * 16 * NB; o += kStreamThreads) {
        const int row = o / (16 * NB), col = o % (16 * NB), r = rb * 16 * NB + col;
        if (!((same >> row) & 1) || r >= a.rank_pad)
            continue;
        const float v = s * stream_sum<MB, NB>(red, row, col);
        if (a.planes) {
            const size_t at = (size_t)(m0 + row) * a.rank_pad + r;
            const __bf16 hi = (__bf16)v;
            ((__bf16 *)a.v)[at] = hi;
            ((__bf16 *)a.v)[(size_t)a.M * a.rank_pad + at] = (__bf16)(v - (float)hi);
        } else {
            ((float *)a.v)[((size_t)part * a.M + m0 + row) * a.rank_pad + r] = v;
        }
    }
}

__device__ inline int row_id(const LoraArgs &a, bool there, int row)
{
    const int id = there ? a.adapter[row] : -1;
    return (uint32_t)id < (uint32_t)a.adapters ? id : -1;
}

}  // namespace

__global__ __launch_bounds__(kStreamThreads, 4) void lora_down_few_kernel(const LoraArgs a)
{
    __shared__ float red[kStreamWaves][16][stream_pitch<1>()];
    const int m0 = blockIdx.x * 16, l = lane_id();
    const int rb = blockIdx.z / a.parts, part = blockIdx.z - rb * a.parts;
    unsigned long long same = 0;
    const int e = lora_nth(row_id(a, l < 16 && m0 + l < a.M, m0 + l), ~0ull, blockIdx.y, &same);
    if (e >= 0)
        lora_down<1, 1>(a, m0, e, same, rb, part, red);
}

// Workgroups 0 .. blocks - 1: the first adapter of each block of 16 MB rows.
// The rest: kLoraMore per group of 64 rows, for the groups' further adapters.
template <int MB, int NB>
__global__ __launch_bounds__(kStreamThreads, 2) void lora_down_many_kernel(const LoraArgs a, int blocks)
{
    __shared__ float red[kStreamWaves][16 * MB][stream_pitch<NB>()];
    const int l = lane_id(), rb = blockIdx.y;
    if ((int)blockIdx.x < blocks) {
        const int m0 = blockIdx.x * 16 * MB;
        unsigned long long same = 0;
        const int e = lora_nth(row_id(a, l < 16 * MB && m0 + l < a.M, m0 + l), ~0ull, 0, &same);
        if (e >= 0)
            lora_down<MB, NB>(a, m0, e, same, rb, 0, red);
        return;
    }
    const int more = (int)blockIdx.x - blocks, g = more / kLoraMore, mine = more - g * kLoraMore;
    const int id = row_id(a, g * 64 + l < a.M, g * 64 + l);
    int k = 0;
    for (int b = 0; b < 4 / MB; ++b) {
        const unsigned long long mask = ((MB == 1 ? 0xFFFFull : 0xFFFFFFFFull)) << (16 * MB * b);
        for (int n = 1;; ++n) {
            unsigned long long same = 0;
            const int e = lora_nth(id, mask, n, &same);
            if (e < 0)
                break;
            if (k++ % kLoraMore != mine)
                continue;
            lora_down<MB, NB>(a, g * 64 + 16 * MB * b, e, same >> (16 * MB * b), rb, 0, red);
            __syncthreads();
        }
    }
}

namespace {

template <int MB, int NB>
hipError_t many(const LoraArgs &a, int passes, hipStream_t s)
{
    const int64_t blocks = ((int64_t)a.M + 16 * MB - 1) / (16 * MB);
    const int64_t more = a.adapters > 1 ? ((int64_t)a.M + 63) / 64 * kLoraMore : 0;
    hipLaunchKernelGGL((lora_down_many_kernel<MB, NB>), dim3((unsigned)(blocks + more), (unsigned)passes),
                       dim3(kStreamThreads), 0, s, a, (int)blocks);
    return hipGetLastError();
}

template <int MB>
hipError_t many_mb(const LoraArgs &a, int blocks, hipStream_t s)
{
    if (blocks == 2)                                 // (rank_pad is a multiple of 32)
        return many<MB, 2>(a, 1, s);
    return many<MB, 4>(a, (blocks + 3) / 4, s);
}

}  // namespace

hipError_t launch_lora_down(const LoraArgs &a, hipStream_t s)
{
    const int blocks = a.rank_pad / 16;
    if (a.M <= kLoraFewRows) {
        const unsigned rows = (unsigned)((a.M + 15) / 16);
        hipLaunchKernelGGL(lora_down_few_kernel,
                           dim3(rows, (unsigned)(a.adapters < 16 ? a.adapters : 16), (unsigned)(blocks * a.parts)),
                           dim3(kStreamThreads), 0, s, a);
        return hipGetLastError();
    }
    return a.M <= 8192 ? many_mb<1>(a, blocks, s) : many_mb<2>(a, blocks, s);
}

}  // namespace tg
