// Low-rank adapters of many requests, the first half:
//
//   v[m][r] = s_a sum_k x[m][k] down_a[r][k],     a the adapter of row m
//
// in fp32, for the projection's kernel to finish (lora.hpp).  Two forms of one
// kernel, by the number of rows:
//   * up to kLoraFewRows (decode): the adapters' matrices are the bytes, most
//     rows have one of their own, and a workgroup alone would take long over
//     one.  So a workgroup takes one adapter of 16 rows, 16 of its ranks and one
//     part of K; the parts are added by the reader.
//   * above (prompts, training): x is the bytes.  A workgroup takes 16 or 32
//     rows with up to 64 ranks at once, x read once for them, and one adapter
//     after the other where its rows have several.
#include "stream.hpp"

namespace tg {

namespace {

// The n-th adapter (in the order of its first row) among up to 64 rows, or -1;
// same: its rows.  id: one row per lane, -1 without an adapter.
__device__ inline int lora_nth(int id, int n, unsigned long long *same)
{
    unsigned long long left = __ballot(id >= 0);
    while (left) {
        const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        *same = __ballot(id == e);
        if (n-- == 0)
            return e;
        left &= ~*same;
    }
    return -1;
}

}  // namespace

// Rows 16 MB blockIdx.x .., ranks 16 NB rank_block .., K steps of part `part`.
// FEW: only the blockIdx.y-th adapter of the rows; else all of them.
template <int MB, int NB, bool FEW>
__global__ __launch_bounds__(kStreamThreads, FEW ? 4 : 2) void lora_down_kernel(const LoraArgs a)
{
    __shared__ float red[kStreamWaves][16 * MB][stream_pitch<NB>()];
    const int l = lane_id(), r16 = l & 15;
    const int m0 = blockIdx.x * 16 * MB;
    const int rb = blockIdx.z / a.parts, part = blockIdx.z - rb * a.parts;
    const int row = m0 + l;
    int id = l < 16 * MB && row < a.M ? a.adapter[row] : -1;
    id = (uint32_t)id < (uint32_t)a.adapters ? id : -1;
    const uint32_t kb = (uint32_t)a.K * 2u;
    const int steps = (int)(kb / 64), per = (steps + a.parts - 1) / a.parts;
    const int step0 = min(part * per, steps), n_steps = min(per, steps - step0);
    const auto rX = make_rsrc((const uint8_t *)a.x + (size_t)m0 * kb, (uint32_t)min(a.M - m0, 16 * MB) * kb);
    uint32_t xoff[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
        xoff[i] = keep_or_oob(m0 + i * 16 + r16 < a.M, (uint32_t)(i * 16 + r16) * kb);
    float *const v = a.v_out + (size_t)part * a.M * a.rank_pad;
    for (int n = FEW ? (int)blockIdx.y : 0;; ++n) {
        unsigned long long same = 0;
        const int e = lora_nth(id, n, &same);
        if (e < 0)
            return;
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
            const int orow = o / (16 * NB), col = o % (16 * NB), r = rb * 16 * NB + col;
            if (((same >> orow) & 1) && r < a.rank_pad)
                v[(size_t)(m0 + orow) * a.rank_pad + r] = s * stream_sum<MB, NB>(red, orow, col);
        }
        if (FEW)
            return;
        __syncthreads();
    }
}

namespace {

template <int MB, int NB, bool FEW>
hipError_t launch(const LoraArgs &a, dim3 grid, hipStream_t s)
{
    hipLaunchKernelGGL((lora_down_kernel<MB, NB, FEW>), grid, dim3(kStreamThreads), 0, s, a);
    return hipGetLastError();
}

template <int MB>
hipError_t launch_many(const LoraArgs &a, int blocks, hipStream_t s)
{
    const unsigned rows = (unsigned)((a.M + 16 * MB - 1) / (16 * MB));
    if (blocks == 1)
        return launch<MB, 1, false>(a, dim3(rows), s);
    if (blocks == 2)
        return launch<MB, 2, false>(a, dim3(rows), s);
    return launch<MB, 4, false>(a, dim3(rows, 1, (unsigned)((blocks + 3) / 4)), s);
}

}  // namespace

hipError_t launch_lora_down(const LoraArgs &a, hipStream_t s)
{
    const int blocks = a.rank_pad / 16;
    if (a.M <= kLoraFewRows) {
        const unsigned rows = (unsigned)((a.M + 15) / 16);
        return launch<1, 1, true>(a, dim3(rows, (unsigned)(a.adapters < 16 ? a.adapters : 16), (unsigned)(blocks * a.parts)), s);
    }
    return a.M <= 8192 ? launch_many<1>(a, blocks, s) : launch_many<2>(a, blocks, s);
}

}  // namespace tg
