// A whole mixture-of-experts layer for a few tokens, in two launches:
//
//   h[s]   = act(x[t] G_e^T) * (x[t] U_e^T)      slot s = t topk + j, e = ids[s]    (or act(x[t] U_e^T))
//   out[t] = sum over j of w[s] (h[s] D_e^T)  (+ residual[t])
//
// Bound: HBM, by the weights of the active experts, each read once.  What is
// left to the design is to keep enough of them in flight from the first
// microsecond to the last:
//   * no routing tables from a launch before: every workgroup marks the active
//     experts in an LDS bitmap by itself (ids are a few KiB at most) and picks
//     its work by counting bits;
//   * the launch is two workgroups per CU, which walk the items (active
//     expert, column tile), so nothing is launched for experts nobody chose;
//   * an item's 32 weight rows (16 of the gate and the 16 of the linear half
//     that meet them, or 32 columns of the output) are read straight into
//     registers in MFMA order, the waves splitting K, each with two sets of
//     loads in flight; the tokens' rows come from the caches;
//   * the second launch's sums over experts meet in the workspace: each item
//     writes its slots' fp32 sums, and the workgroup that finishes a column tile
//     last adds the slots of every token in the order of j.  Which workgroup that
//     is does not change the result.
#include "stream.hpp"

namespace tg {

namespace {

constexpr int kMlpThreads = kStreamThreads;
constexpr int kMlpPitch = stream_pitch<2>();
constexpr int kMlpBits = kMaxGroups / 32;          // words of the bitmap of experts
static_assert(kMlpBits == 32, "one word per lane of half a wave");

// What every workgroup knows of the routing.
struct MlpShared {
    uint32_t bits[kMlpBits];
    uint16_t ids[kMlpSlots];         // 0xFFFF: a slot that goes nowhere
    uint16_t rows[kMlpSlots];        // the current expert's slots, in order
    int32_t cnt;
    int32_t last;
};

// Marks the experts that some slot names.  Returns their number.
__device__ inline int mlp_mark(MlpShared &sh, const MlpArgs &a)
{
    if (threadIdx.x < kMlpBits)
        sh.bits[threadIdx.x] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < a.slots; s += kMlpThreads) {
        const int id = a.ids[s];
        const bool in = (uint32_t)id < (uint32_t)a.groups;
        sh.ids[s] = in ? (uint16_t)id : (uint16_t)0xFFFF;
        if (in)
            atomicOr(&sh.bits[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    const int l = lane_id();
    int n = l < kMlpBits ? __popc(sh.bits[l & (kMlpBits - 1)]) : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        n += __shfl_xor(n, d);
    return __builtin_amdgcn_readfirstlane(n);
}

// The p-th active expert (p below their number), in increasing order.
__device__ inline int mlp_expert(const MlpShared &sh, int p)
{
    const int l = lane_id();
    const uint32_t word = l < kMlpBits ? sh.bits[l & (kMlpBits - 1)] : 0u;
    int x = __popc(word);
    const int n = x;
#pragma unroll
    for (int d = 1; d < kMlpBits; d <<= 1) {
        const int y = __shfl_up(x, d);
        x += l >= d ? y : 0;
    }
    const int lane = __builtin_ctzll(__ballot(x > p));
    uint32_t w = __builtin_amdgcn_readlane(word, lane);
    for (int skip = p - __builtin_amdgcn_readlane(x - n, lane); skip > 0; --skip)
        w &= w - 1;
    return __builtin_amdgcn_readfirstlane(lane * 32 + __builtin_ctz(w));
}

// The slots of expert e into sh.rows, in order.
__device__ inline int mlp_rows(MlpShared &sh, int slots, int e)
{
    __syncthreads();                                 // the previous expert's rows are no longer read
    if (wave_id() == 0) {
        const int l = lane_id();
        const unsigned long long below = (1ull << l) - 1;
        int n = 0;
        for (int s0 = 0; s0 < slots; s0 += 64) {
            const bool mine = s0 + l < slots && sh.ids[s0 + l] == e;
            const unsigned long long m = __ballot(mine);
            if (mine)
                sh.rows[n + __popcll(m & below)] = (uint16_t)(s0 + l);
            n += __popcll(m);
        }
        if (l == 0)
            sh.cnt = n;
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(sh.cnt);
}

}  // namespace

// x -> h.  Column tile c: the gate's and the linear half's columns 16 c .. + 15
// (GATED), or columns 32 c .. + 31.
template <int MB, bool E8, bool PRE, int U>
__device__ inline void mlp_up_item(const MlpArgs &a, const MlpShared &sh, int e, int r0, int cnt, int c, float *lds)
{
    float(*red)[16 * MB][kMlpPitch] = reinterpret_cast<float(*)[16 * MB][kMlpPitch]>(lds);
    const int r16 = lane_id() & 15;
    const uint32_t kb = (uint32_t)a.K * (E8 ? 1u : 2u);
    const int inner = a.gated ? 2 * a.N : a.N;
    const int n0 = a.gated ? 16 * c : 32 * c, n1 = a.gated ? a.N + 16 * c : 32 * c + 16;
    const uint8_t *const W = (const uint8_t *)a.up + (size_t)e * inner * kb;
    const __amdgpu_buffer_rsrc_t rB[2] = {make_rsrc(W + (size_t)n0 * kb, 16u * kb),
                                          make_rsrc(W + (size_t)n1 * kb, 16u * kb)};
    const auto rX = make_rsrc(a.x, (uint32_t)a.tokens * (uint32_t)a.K * 2u);
    uint32_t xoff[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int r = r0 + i * 16 + r16;
        xoff[i] = keep_or_oob(r < cnt, (uint32_t)(sh.rows[r < cnt ? r : 0] / a.topk) * (uint32_t)a.K * 2u);
    }
    stream_product<MB, 2, E8, PRE, U>(rX, xoff, rB, kb, 0, (int)(kb / 64), red);
    __syncthreads();
    const int cols = a.gated ? 16 : 32;
    for (int o = threadIdx.x; o < 16 * MB * cols; o += kMlpThreads) {
        const int row = o / cols, col = o - row * cols;
        const int n = n0 + col;
        if (r0 + row >= cnt)
            continue;
        const size_t at = (size_t)e * inner + n;
        float z = stream_sum<MB, 2>(red, row, col);
        if (a.up_scale)
            z *= a.up_scale[at];
        if (a.up_bias)
            z += a.up_bias[at];
        float y = a.act == kActSilu ? epi_silu(z) : epi_act(z, a.act);
        if (a.gated) {
            float u = stream_sum<MB, 2>(red, row, 16 + col);
            if (a.up_scale)
                u *= a.up_scale[at + a.N];
            if (a.up_bias)
                u += a.up_bias[at + a.N];
            y *= u;
        }
        // h in bf16: the second product's operand, as the layer made of
        // single products keeps it
        ((__bf16 *)a.h)[(size_t)sh.rows[r0 + row] * a.N + n] = (__bf16)y;
    }
}

template <int MB, bool E8, bool PRE>
__global__ __launch_bounds__(kMlpThreads, 4) void mlp_up_kernel(const MlpArgs a)
{
    __shared__ MlpShared sh;
    __shared__ float lds[kStreamWaves * 16 * MB * kMlpPitch];
    constexpr int U = E8 ? 2 : 4;
    if (blockIdx.x == 0)
        for (int c = threadIdx.x; c < a.down_tiles; c += kMlpThreads)
            a.done[c] = 0;
    const int active = mlp_mark(sh, a), items = active * a.up_tiles;
    int p = -1, e = 0, cnt = 0;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int np = it / a.up_tiles, c = it - np * a.up_tiles;
        if (np != p) {
            p = np;
            e = mlp_expert(sh, p);
            cnt = mlp_rows(sh, a.slots, e);
        }
        for (int r0 = 0; r0 < cnt; r0 += 16 * MB) {
            if (MB == 1 || cnt - r0 <= 16)
                mlp_up_item<1, E8, PRE, U>(a, sh, e, r0, cnt, c, lds);
            else
                mlp_up_item<MB, E8, PRE, U / 2>(a, sh, e, r0, cnt, c, lds);
            __syncthreads();                         // the sums have been read
        }
    }
}

// h -> the slots' sums, columns 32 c .. + 31 of the output.
template <int MB, bool E8, bool PRE, int U>
__device__ inline void mlp_down_item(const MlpArgs &a, const MlpShared &sh, int e, int r0, int cnt, int c, float *lds)
{
    float(*red)[16 * MB][kMlpPitch] = reinterpret_cast<float(*)[16 * MB][kMlpPitch]>(lds);
    const int r16 = lane_id() & 15;
    const uint32_t kb = (uint32_t)a.N * (E8 ? 1u : 2u);
    const int n0 = 32 * c;
    const uint8_t *const W = (const uint8_t *)a.down + (size_t)e * a.K * kb;
    const __amdgpu_buffer_rsrc_t rB[2] = {make_rsrc(W + (size_t)n0 * kb, 16u * kb),
                                          make_rsrc(W + (size_t)(n0 + 16) * kb, 16u * kb)};
    const auto rX = make_rsrc(a.h, (uint32_t)a.slots * (uint32_t)a.N * 2u);
    uint32_t xoff[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int r = r0 + i * 16 + r16;
        xoff[i] = keep_or_oob(r < cnt, (uint32_t)sh.rows[r < cnt ? r : 0] * (uint32_t)a.N * 2u);
    }
    stream_product<MB, 2, E8, PRE, U>(rX, xoff, rB, kb, 0, (int)(kb / 64), red);
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * MB * 32; o += kMlpThreads) {
        const int row = o / 32, n = n0 + o % 32;
        if (r0 + row >= cnt)
            continue;
        const size_t at = (size_t)e * a.K + n;
        float z = stream_sum<MB, 2>(red, row, o % 32);
        if (a.down_scale)
            z *= a.down_scale[at];
        if (a.down_bias)
            z += a.down_bias[at];
        __hip_atomic_store(a.y + (size_t)sh.rows[r0 + row] * a.K + n, z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

template <int MB, bool E8, bool PRE>
__global__ __launch_bounds__(kMlpThreads, 4) void mlp_down_kernel(const MlpArgs a)
{
    __shared__ MlpShared sh;
    __shared__ float lds[kStreamWaves * 16 * MB * kMlpPitch];
    constexpr int U = E8 ? 2 : 4;
    // Without any active expert the column tiles still have to be written.
    const int active = mlp_mark(sh, a), parts = max(active, 1), items = parts * a.down_tiles;
    int p = -1, e = 0, cnt = 0;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int np = it / a.down_tiles, c = it - np * a.down_tiles;
        if (active && np != p) {
            p = np;
            e = mlp_expert(sh, p);
            cnt = mlp_rows(sh, a.slots, e);
        }
        for (int r0 = 0; r0 < cnt; r0 += 16 * MB) {
            if (MB == 1 || cnt - r0 <= 16)
                mlp_down_item<1, E8, PRE, U>(a, sh, e, r0, cnt, c, lds);
            else
                mlp_down_item<MB, E8, PRE, U / 2>(a, sh, e, r0, cnt, c, lds);
            __syncthreads();
        }
        // This item's sums are out before it counts as done; the last one of
        // the column tile sees all of them.  The XCDs' L2 caches are not
        // coherent with each other, so the sums are written through and read
        // past them (agent scope on each access), and waiting for the stores
        // is all a release has to do.  With a release fence instead, which
        // writes the whole L2 back for every wave, the launch took 88 us for one
        // token and 652 us for 16.
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0)
            sh.last = __hip_atomic_fetch_add(&a.done[c], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
        __syncthreads();
        if (!sh.last)
            continue;
        asm volatile("" ::: "memory");
        for (int o = threadIdx.x; o < a.tokens * 32; o += kMlpThreads) {
            const int t = o / 32, n = 32 * c + o % 32;
            float sum = 0.f;
#pragma unroll 4
            for (int j = 0; j < a.topk; ++j) {
                const int s = t * a.topk + j;
                if (sh.ids[s] == 0xFFFF)
                    continue;                        // nor is its weight read as a factor
                const float y = __hip_atomic_load(a.y + (size_t)s * a.K + n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                sum = fmaf(a.weights ? a.weights[s] : 1.f, y, sum);
            }
            const size_t at = (size_t)t * a.K + n;
            if (a.residual)
                sum += (float)((const __bf16 *)a.residual)[at];
            ((__bf16 *)a.out)[at] = (__bf16)sum;
        }
    }
}

namespace {

template <int MB, bool E8, bool PRE>
hipError_t launch(const MlpArgs &a, hipStream_t s)
{
    const int64_t up = (int64_t)a.parts * a.up_tiles, down = (int64_t)a.parts * a.down_tiles;
    hipLaunchKernelGGL((mlp_up_kernel<MB, E8, PRE>), dim3((unsigned)(up < kMlpGrid ? up : kMlpGrid)),
                       dim3(kMlpThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((mlp_down_kernel<MB, E8, PRE>), dim3((unsigned)(down < kMlpGrid ? down : kMlpGrid)),
                       dim3(kMlpThreads), 0, s, a);
    return hipGetLastError();
}

template <int MB>
hipError_t launch_mb(const MlpArgs &a, hipStream_t s)
{
    if (a.e4m3)
        return a.preshuffled ? launch<MB, true, true>(a, s) : launch<MB, true, false>(a, s);
    return a.preshuffled ? launch<MB, false, true>(a, s) : launch<MB, false, false>(a, s);
}

}  // namespace

hipError_t launch_mlp(const MlpArgs &a, hipStream_t s)
{
    // Up to 16 tokens an expert has one block of rows (unless a token names it
    // more than once, which the loop over its rows takes care of).
    return a.tokens <= 16 ? launch_mb<1>(a, s) : launch_mb<2>(a, s);
}

}  // namespace tg
