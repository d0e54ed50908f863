// A whole mixture-of-experts layer for a few tokens, in two launches:
//
//   h[s]   = act(x[t] G_e^T) * (x[t] U_e^T)      slot s = t topk + j, e = ids[s]    (or act(x[t] U_e^T))
//   out[t] = sum over j of w[s] (h[s] D_e^T)  (+ residual[t])
//
// Bound: HBM, by the weights of the active experts, each read once per 32 rows of
// its expert (16 up to 16 tokens): a pass holds no more, and the next one streams
// them again, mostly from HBM (64 tokens x 2 of 2 experts, 4096 x 2048 gated bf16,
// pre-shuffled: 132 + 50 MiB fetched for 64 + 32, 51.6 us where once takes 19; x 4 of
// 8 with up to 36 rows each 139 us, 171 as they are, once 76).  What is
// left to the design is to keep enough of them in flight from the first
// microsecond to the last:
//   * no routing tables from a launch before: every workgroup marks the active
//     experts in an LDS bitmap by itself (ids are a few KiB at most) and picks
//     its work by counting bits;
//   * the launch is two workgroups per CU, which walk the items (active
//     expert, column tile), so nothing is launched for experts nobody chose;
//   * an item's 32 weight rows (16 of the gate and the 16 of the linear half that
//     meet them, or 32 columns of the output) are read straight into registers
//     in MFMA order, the waves splitting K, each with two sets of loads in
//     flight; the tokens' rows come from the caches, once per item (items of 64
//     weight rows, which halve that, measured 2% faster to 10% slower);
//   * the second launch's sums over experts meet in the workspace: each item
//     writes its slots' fp32 sums, and the workgroup that finishes a column tile
//     last adds the slots of every token in the order of j.  Which workgroup that
//     is does not change the result.
// Measured, both launches: 16 tokens x 4 of 64 experts, 2048 x 1024 gated bf16,
// pre-shuffled: 90 to 99 us, 5.2 to 5.7 TB/s of 518 MB, a copy's rate.  One token x 8:
// 26 us (101 MB, 3.8 TB/s: each launch is one or two items per workgroup, start
// and end included).  61 tokens x 4 of 24, 4096 x 2112 e4m3 as it is: 168 to 177 us,
// 3.5 to 3.7 TB/s: x and h are read once per item, as many bytes again as the 8-bit
// weights (without those reads 146 us).
#include "stream.hpp"

namespace tg {

namespace {

constexpr int kMlpThreads = kStreamThreads;
constexpr int kMlpRows = 32;                       // rows of a pass, at most
constexpr int kMlpBits = kMaxGroups / 32;          // words of the bitmap of experts
static_assert(kMlpBits == 32, "one word per lane of half a wave");

// What every workgroup knows of the routing.
struct MlpShared {
    uint32_t bits[kMlpBits];
    uint16_t ids[kMlpSlots];                     // 0xFFFF: a slot that goes nowhere
    uint16_t rows[kStreamWaves][kMlpRows];       // each wave's own copy of the slots of the rows at hand
    int32_t last[2];                             // of the passes in turn: read behind a barrier, written before the next
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

// Rows r0 .. r0 + kMlpRows - 1 of expert e (its slots, in order) into this wave's
// list.  Returns the number of all its rows.  Every wave looks for itself, so
// nothing has to be waited for.
__device__ inline int mlp_rows(MlpShared &sh, int slots, int e, int r0)
{
    const int l = lane_id();
    uint16_t *const rows = sh.rows[wave_id()];
    const unsigned long long below = (1ull << l) - 1;
    int n = 0;
    for (int s0 = 0; s0 < slots; s0 += 64) {
        const bool mine = s0 + l < slots && sh.ids[s0 + l] == e;
        const unsigned long long m = __ballot(mine);
        const int at = n + __popcll(m & below) - r0;
        if (mine && at >= 0 && at < kMlpRows)
            rows[at] = (uint16_t)(s0 + l);
        n += __popcll(m);
    }
    __builtin_amdgcn_wave_barrier();
    return __builtin_amdgcn_readfirstlane(n);
}

// LDS of the waves' sums: two sets, so that one barrier per pass is enough (a
// wave may start on the next pass's products while others still add up this
// one's).
template <int MB>
constexpr int mlp_red() { return kStreamWaves * 16 * MB * stream_pitch<2>(); }

// Steps per set of loads (stream.hpp).  Two sets of two per wave keep 128 KiB in
// flight on a CU, twice what the latency asks for.  Measured, us for 1 / 2 / 3 / 4, 16
// tokens x 4 of 64, 2048 x 1024: up 64 / 61 / 66 / 71, down 38 / 37 / 38 / 46 in bf16;
// up 36 / 35 / 52 / 101, down 27 / 32 / 43 / 96 in e4m3 (whose steps hold twice the K,
// and whose second product leaves a wave only two or so).
template <int MB, bool E8, bool DOWN>
constexpr int mlp_u() { return MB == 1 && !(E8 && DOWN) ? 2 : 1; }

// A workgroup's first item.  Workgroups go to the XCDs in turn; of every 256 the 32
// of an XCD take neighbouring items, mostly of one expert, whose rows of x its L2
// then fetches once.  (Against items in the workgroups' order: 16 tokens x 4 of 64,
// 2048 x 1024 bf16, pre-shuffled 103 -> 99 us, 64 x 8 as they are 198 -> 189.  With 64 of
// 512 in a row, so that the two workgroups of a CU are neighbours as well: 104 and
// 194.)
__device__ inline int mlp_first()
{
    constexpr int kXcds = 8, kRun = 32, kAll = kXcds * kRun;
    const int b = blockIdx.x, c = b % kAll, at = b - c;
    return at + kAll > (int)gridDim.x ? b : at + (c % kXcds) * kRun + c / kXcds;
}

}  // namespace

// x -> h, rows r0 .. of expert e.  Column tile c: the gate's and the linear half's
// columns 16 c .. + 15 (gated), or columns 32 c .. + 31.
template <int MB, bool E8, bool PRE>
__device__ inline void mlp_up_pass(const MlpArgs &a, const MlpShared &sh, int e, int r0, int cnt, int c, float *lds)
{
    float(*red)[16 * MB][stream_pitch<2>()] = reinterpret_cast<float(*)[16 * MB][stream_pitch<2>()]>(lds);
    const uint16_t *const rows = sh.rows[wave_id()];
    const int r16 = lane_id() & 15;
    const uint32_t kb = (uint32_t)a.K * (E8 ? 1u : 2u);
    const int inner = a.gated ? 2 * a.N : a.N;
    const int cols = a.gated ? 16 : 32, n0 = c * cols;
    const uint8_t *const W = (const uint8_t *)a.up + (size_t)e * inner * kb;
    const int n1 = a.gated ? a.N + n0 : n0 + 16;
    auto find = [&](__amdgpu_buffer_rsrc_t (&rB)[2]) {
        rB[0] = make_rsrc(W + (size_t)n0 * kb, 16u * kb);
        rB[1] = make_rsrc(W + (size_t)n1 * kb, 16u * kb);
    };
    const auto rX = make_rsrc(a.x, (uint32_t)a.tokens * (uint32_t)a.K * 2u);
    uint32_t xoff[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int r = i * 16 + r16;
        const bool there = r0 + r < cnt;
        xoff[i] = keep_or_oob(there, (uint32_t)(rows[there ? r : 0] / a.topk) * (uint32_t)a.K * 2u);
    }
    stream_product<MB, 2, E8, PRE, mlp_u<MB, E8, false>()>(rX, xoff, find, kb, 0, (int)(kb / 64), red);
    __syncthreads();
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
            float u = stream_sum<MB, 2>(red, row, cols + col);
            if (a.up_scale)
                u *= a.up_scale[at + a.N];
            if (a.up_bias)
                u += a.up_bias[at + a.N];
            y *= u;
        }
        // h in bf16: the second product's operand, as the layer made of
        // single products keeps it (half the bytes and half the MFMAs of two
        // bf16 numbers).  Against an h in fp32 the output's error grows from
        // 1.7e-3 of its norm, its own rounding, to 1.8e-3 (16 x 4 of 64, with a
        // residual) or 2.2e-3 (61 x 4 of 24, without).
        ((__bf16 *)a.h)[(size_t)rows[row] * a.N + n] = (__bf16)y;
    }
}

template <int MB, bool E8, bool PRE>
__global__ __launch_bounds__(kMlpThreads, 4) void mlp_up_kernel(const MlpArgs a)
{
    __shared__ MlpShared sh;
    __shared__ float lds[2][mlp_red<MB>()];
    if (blockIdx.x == 0)
        for (int c = threadIdx.x; c < a.down_tiles; c += kMlpThreads)
            a.done[c] = 0;
    const int active = mlp_mark(sh, a), items = active * a.up_tiles;
    int set = 0;
    for (int it = mlp_first(); it < items; it += gridDim.x) {
        const int p = it / a.up_tiles, c = it - p * a.up_tiles;
        const int e = mlp_expert(sh, p);
        for (int r0 = 0, cnt = 1; r0 < cnt; r0 += 16 * MB) {
            cnt = mlp_rows(sh, a.slots, e, r0);
            if (MB == 1 || cnt - r0 <= 16)
                mlp_up_pass<1, E8, PRE>(a, sh, e, r0, cnt, c, lds[set]);
            else
                mlp_up_pass<MB, E8, PRE>(a, sh, e, r0, cnt, c, lds[set]);
            set ^= 1;
        }
    }
}

// h -> the slots' sums, column tile c of the output, in two halves: the
// waves' products, and behind the barrier their sum.
template <int MB, bool E8, bool PRE>
__device__ inline void mlp_down_product(const MlpArgs &a, const MlpShared &sh, int e, int r0, int cnt, int c, float *lds)
{
    float(*red)[16 * MB][stream_pitch<2>()] = reinterpret_cast<float(*)[16 * MB][stream_pitch<2>()]>(lds);
    const uint16_t *const rows = sh.rows[wave_id()];
    const int r16 = lane_id() & 15;
    const uint32_t kb = (uint32_t)a.N * (E8 ? 1u : 2u);
    const uint8_t *const W = (const uint8_t *)a.down + ((size_t)e * a.K + 32 * c) * kb;
    auto find = [&](__amdgpu_buffer_rsrc_t (&rB)[2]) {
        rB[0] = make_rsrc(W, 16u * kb);
        rB[1] = make_rsrc(W + (size_t)16 * kb, 16u * kb);
    };
    const auto rX = make_rsrc(a.h, (uint32_t)a.slots * (uint32_t)a.N * 2u);
    uint32_t xoff[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int r = i * 16 + r16;
        const bool there = r0 + r < cnt;
        xoff[i] = keep_or_oob(there, (uint32_t)rows[there ? r : 0] * (uint32_t)a.N * 2u);
    }
    stream_product<MB, 2, E8, PRE, mlp_u<MB, E8, true>()>(rX, xoff, find, kb, 0, (int)(kb / 64), red);
}

template <int MB>
__device__ inline void mlp_down_sum(const MlpArgs &a, const MlpShared &sh, int e, int r0, int cnt, int c, const float *lds)
{
    const float(*red)[16 * MB][stream_pitch<2>()] = reinterpret_cast<const float(*)[16 * MB][stream_pitch<2>()]>(lds);
    const uint16_t *const rows = sh.rows[wave_id()];
    for (int o = threadIdx.x; o < 16 * MB * 32; o += kMlpThreads) {
        const int row = o / 32, n = 32 * c + o % 32;
        if (r0 + row >= cnt)
            continue;
        const size_t at = (size_t)e * a.K + n;
        float z = stream_sum<MB, 2>(red, row, o % 32);
        if (a.down_scale)
            z *= a.down_scale[at];
        if (a.down_bias)
            z += a.down_bias[at];
        __hip_atomic_store(a.y + (size_t)rows[row] * a.K + n, z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// Column tile c of the output, from its slots' sums.
__device__ inline void mlp_combine(const MlpArgs &a, const MlpShared &sh, int c)
{
    for (int o = threadIdx.x; o < a.tokens * 32; o += kMlpThreads) {
        const int t = o / 32, n = 32 * c + o % 32;
        float sum = 0.f;
#pragma unroll 4
        for (int j = 0; j < a.topk; ++j) {
            const int s = t * a.topk + j;
            if (sh.ids[s] == 0xFFFF)
                continue;                            // nor is its weight read as a factor
            const float y = __hip_atomic_load(a.y + (size_t)s * a.K + n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            sum = fmaf(a.weights ? a.weights[s] : 1.f, y, sum);
        }
        const size_t at = (size_t)t * a.K + n;
        if (a.residual)
            sum += (float)((const __bf16 *)a.residual)[at];
        ((__bf16 *)a.out)[at] = (__bf16)sum;
    }
}

// An item's sums have to be out before it counts as done, and the workgroup
// that counts a column tile's last item adds them up.  The XCDs' L2 caches are
// not coherent with each other, so the sums are written through and read past
// them (agent scope on each access), and waiting for the stores is all a
// release has to do.  With a release fence instead, which writes the whole L2
// back for every wave, the launch took 88 us for one token and 652 us for 16.
//
// Neither the stores nor the counter's reply are waited for where they are
// issued: a pass first runs the products of the next item, and what went out in
// the pass before has long arrived by then.  `stored`: the column tile whose last
// sums the previous pass stored; `counted`: the one whose counter it raised, the
// reply in `reply` (thread 0).
template <int MB, bool E8, bool PRE>
__global__ __launch_bounds__(kMlpThreads, 4) void mlp_down_kernel(const MlpArgs a)
{
    __shared__ MlpShared sh;
    __shared__ float lds[2][mlp_red<MB>()];
    // Without any active expert the column tiles still have to be written.
    const int active = mlp_mark(sh, a), parts = max(active, 1), items = parts * a.down_tiles;
    int it = mlp_first(), r0 = 0, set = 0, stored = -1, counted = -1, reply = 0, turn = 0;
    while (it < items || stored >= 0 || counted >= 0) {
        int p = 0, c = -1, e = 0, cnt = 0;
        if (it < items) {
            p = it / a.down_tiles;
            c = it - p * a.down_tiles;
            if (active) {
                e = mlp_expert(sh, p);
                cnt = mlp_rows(sh, a.slots, e, r0);
                if (MB == 1 || cnt - r0 <= 16)
                    mlp_down_product<1, E8, PRE>(a, sh, e, r0, cnt, c, lds[set]);
                else
                    mlp_down_product<MB, E8, PRE>(a, sh, e, r0, cnt, c, lds[set]);
            }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // the previous pass's sums are out
        if (threadIdx.x == 0)
            sh.last[turn] = counted >= 0 && reply == parts - 1;
        __syncthreads();
        const int ready = sh.last[turn] ? counted : -1;
        turn ^= 1;
        counted = stored;
        if (threadIdx.x == 0 && stored >= 0)
            reply = __hip_atomic_fetch_add(&a.done[stored], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        stored = -1;
        if (c >= 0) {
            if (MB == 1 || cnt - r0 <= 16)
                mlp_down_sum<1>(a, sh, e, r0, cnt, c, lds[set]);
            else
                mlp_down_sum<MB>(a, sh, e, r0, cnt, c, lds[set]);
            set ^= 1;
            r0 += 16 * MB;
            if (r0 >= cnt) {                                   // the item's last rows
                stored = c;
                it += gridDim.x;
                r0 = 0;
            }
        }
        if (ready >= 0)
            mlp_combine(a, sh, ready);
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
hipError_t launch_tokens(const MlpArgs &a, hipStream_t s)
{
    if (a.e4m3)
        return a.preshuffled ? launch<MB, true, true>(a, s) : launch<MB, true, false>(a, s);
    return a.preshuffled ? launch<MB, false, true>(a, s) : launch<MB, false, false>(a, s);
}

}  // namespace

hipError_t launch_mlp(const MlpArgs &args, hipStream_t s)
{
    MlpArgs a = args;
    a.up_tiles = a.N / (a.gated ? 16 : 32);
    a.down_tiles = a.K / 32;
    // Up to 16 tokens an expert has one block of rows (unless a token names it
    // more than once, which the loop over its rows takes care of).
    return a.tokens <= 16 ? launch_tokens<1>(a, s) : launch_tokens<2>(a, s);
}

}  // namespace tg
