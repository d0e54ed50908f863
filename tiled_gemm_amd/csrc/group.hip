// The memory-bound operators around the grouped products: the routing tables
// (a stable counting sort by expert), the weighted sum of a token's rows and
// its gradient, and the gradient of the fused epilogue.
#include "group.hpp"

namespace tg {

// ---------------------------------------------------------------------------
// Routing tables.  Slot s (of `slots`) carries an expert id; its sorted row is
//   offsets[id] + (slots before s with the same id).
// Slots are cut into blocks of consecutive slots and a block's slots into 16
// consecutive runs, one per wave, taken 64 at a time.  Equal ids inside 64
// slots are found with one ballot per id bit (no atomics: the order, and so
// the result, is the same on every run), a wave's counters live in LDS.
// One launch when one block holds all slots; otherwise a first launch writes
// every block's counts, and each block of the second sums the counts of the
// blocks before it itself, which saves a third launch for the scan.
// ---------------------------------------------------------------------------
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;

// Lanes of the wave whose id equals this lane's; 0 for a lane without an id.
__device__ inline unsigned long long same_id(int id, bool in, int bits)
{
    unsigned long long m = __ballot(in);
    for (int b = 0; b < bits; ++b) {
        const unsigned long long v = __ballot((id >> b) & 1);
        m &= (id >> b) & 1 ? v : ~v;
    }
    return in ? m : 0;
}

}  // namespace

__global__ __launch_bounds__(kSortThreads) void group_count_kernel(const SortArgs a)
{
    __shared__ int32_t count[kMaxGroups];
    for (int g = threadIdx.x; g < a.groups; g += kSortThreads)
        count[g] = 0;
    __syncthreads();
    const int lo = blockIdx.x * a.block_slots, hi = min(lo + a.block_slots, a.slots);
    for (int s = lo + (int)threadIdx.x; s < hi; s += kSortThreads) {
        const int id = a.ids[s];
        if ((uint32_t)id < (uint32_t)a.groups)
            atomicAdd(&count[id], 1);            // integer counts: the order does not matter
    }
    __syncthreads();
    for (int g = threadIdx.x; g < a.groups; g += kSortThreads)
        a.counts[(size_t)blockIdx.x * a.groups + g] = count[g];
}

__global__ __launch_bounds__(kSortThreads) void group_place_kernel(const SortArgs a)
{
    __shared__ int32_t hist[kSortWaves][kMaxGroups];    // per wave: counts, then the next row of each group
    __shared__ int32_t wave_sum[kSortWaves];
    __shared__ int32_t part_total[kSortThreads], part_before[kSortThreads];
    const int tid = threadIdx.x, w = wave_id(), l = lane_id();
    volatile int32_t *mine = hist[w];
    for (int g = l; g < a.groups; g += 64)
        mine[g] = 0;
    const int block_lo = blockIdx.x * a.block_slots;
    const int run = a.block_slots / kSortWaves;           // a multiple of 64
    const int lo = min(block_lo + w * run, a.slots), hi = min(lo + run, a.slots);
    const unsigned long long below = (1ull << l) - 1;
    __builtin_amdgcn_wave_barrier();
    for (int s0 = lo; s0 < hi; s0 += 64) {
        const int s = s0 + l;
        const int id = s < hi ? a.ids[s] : -1;
        const bool in = (uint32_t)id < (uint32_t)a.groups;
        const unsigned long long m = same_id(id, in, a.id_bits);
        if (in && (m & below) == 0)
            mine[id] = mine[id] + __popcll(m);
    }
    __syncthreads();
    // Thread g: group g's rows in all blocks and in the blocks before this one.
    // With several blocks all threads share the reading: thread p * 2^id_bits + g
    // adds up every (1024 / 2^id_bits)-th block from block p on.
    int total = 0, before = 0;
    if (a.blocks > 1) {
        const int wide = 1 << a.id_bits, parts = kSortThreads / wide;
        const int g = tid & (wide - 1), part = tid >> a.id_bits;
        int sum = 0, early = 0;
        if (g < a.groups) {
#pragma unroll 8
            for (int b = part; b < a.blocks; b += parts) {
                const int c = a.counts[(size_t)b * a.groups + g];
                sum += c;
                early += b < (int)blockIdx.x ? c : 0;
            }
        }
        part_total[tid] = sum;
        part_before[tid] = early;
        __syncthreads();
        if (tid < a.groups) {
            for (int i = 0; i < parts; ++i) {
                total += part_total[(i << a.id_bits) + tid];
                before += part_before[(i << a.id_bits) + tid];
            }
        }
    } else if (tid < a.groups) {
        for (int ww = 0; ww < kSortWaves; ++ww)
            total += hist[ww][tid];
    }
    int x = total;                                         // inclusive sum over the groups
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(x, d);
        x += l >= d ? y : 0;
    }
    if (l == 63)
        wave_sum[w] = x;
    __syncthreads();
    int base = x - total;
    for (int ww = 0; ww < w; ++ww)
        base += wave_sum[ww];
    if (tid < a.groups) {
        if (blockIdx.x == 0) {
            a.offsets[tid] = base;
            if (tid == a.groups - 1)
                a.offsets[a.groups] = base + total;
        }
        int next = base + before;
        for (int ww = 0; ww < kSortWaves; ++ww) {
            const int c = hist[ww][tid];
            hist[ww][tid] = next;
            next += c;
        }
    }
    __syncthreads();
    for (int s0 = lo; s0 < hi; s0 += 64) {
        const int s = s0 + l;
        const int id = s < hi ? a.ids[s] : -1;
        const bool in = (uint32_t)id < (uint32_t)a.groups;
        const unsigned long long m = same_id(id, in, a.id_bits);
        int row = -1;
        if (in) {
            row = mine[id] + __popcll(m & below);
            a.row_token[row] = s / a.topk;
        }
        __builtin_amdgcn_wave_barrier();                   // every lane has read its counter
        if (in && (m & below) == 0)
            mine[id] = mine[id] + __popcll(m);
        __builtin_amdgcn_wave_barrier();
        if (s < hi)
            a.slot_row[s] = row;
    }
}

hipError_t launch_group_sort(const SortArgs &a, hipStream_t s)
{
    if (a.blocks > 1) {
        hipLaunchKernelGGL(group_count_kernel, dim3(a.blocks), dim3(kSortThreads), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(group_place_kernel, dim3(a.blocks), dim3(kSortThreads), 0, s, a);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Eight consecutive columns of a bf16 or fp32 row as fp32, and back.
// ---------------------------------------------------------------------------
namespace {

template <int T>
__device__ inline void load8(const void *base, size_t at, float (&v)[8])
{
    if constexpr (T == kOutF32) {
        const f32x4 lo = *(const f32x4 *)((const float *)base + at), hi = *(const f32x4 *)((const float *)base + at + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = lo[i];
            v[4 + i] = hi[i];
        }
    } else {
        const u32x4 w = *(const u32x4 *)((const uint16_t *)base + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}

template <int T>
__device__ inline void store8(void *base, size_t at, const float (&v)[8])
{
    if constexpr (T == kOutF32) {
        *(f32x4 *)((float *)base + at) = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4 *)((float *)base + at + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        *(u32x4 *)((uint16_t *)base + at) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
}

constexpr int kCombineThreads = 256;
// A launch has fewer than 2^32 threads.
constexpr int64_t kCombineBlocks = (int64_t)1 << 23;

}  // namespace

// ---------------------------------------------------------------------------
// out[t] = sum_j weights[t][j] * src[slot_row[t][j]] (+ residual[t]).
// Bound: HBM (every routed row is read once, every token written once).  A
// thread owns 8 columns of one token, so the sum over j is its own, in order.
// ---------------------------------------------------------------------------
template <int T>
__global__ __launch_bounds__(kCombineThreads) void group_combine_kernel(const CombineArgs a)
{
    const int64_t per = a.N / 8, items = a.tokens * per;
    for (int64_t it = (int64_t)blockIdx.x * kCombineThreads + threadIdx.x; it < items;
         it += (int64_t)gridDim.x * kCombineThreads) {
        const int64_t t = it / per;
        const int64_t col = (it - t * per) * 8;
        float sum[8] = {};
        for (int j = 0; j < a.topk; ++j) {
            const int row = a.slot_row[t * a.topk + j];
            if ((uint32_t)row >= (uint32_t)a.src_rows)
                continue;
            const float w = a.weights ? a.weights[t * a.topk + j] : 1.f;
            float v[8];
            load8<T>(a.src, (size_t)row * a.N + col, v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[i] = fmaf(w, v[i], sum[i]);
        }
        if (a.residual) {
            float v[8];
            load8<T>(a.residual, (size_t)t * a.N + col, v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[i] += v[i];
        }
        store8<T>(a.out, (size_t)t * a.N + col, sum);
    }
}

hipError_t launch_group_combine(const CombineArgs &a, hipStream_t s)
{
    const int64_t blocks = (a.tokens * (a.N / 8) + kCombineThreads - 1) / kCombineThreads;
    const unsigned grid = (unsigned)(blocks < kCombineBlocks ? blocks : kCombineBlocks);
    if (a.type == kOutF32)
        hipLaunchKernelGGL(group_combine_kernel<kOutF32>, dim3(grid), dim3(kCombineThreads), 0, s, a);
    else
        hipLaunchKernelGGL(group_combine_kernel<kOutBf16>, dim3(grid), dim3(kCombineThreads), 0, s, a);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// d_src[row(t, j)] = weights[t][j] * d_out[t];  d_weights[t][j] = <d_out[t],
// src[row(t, j)]>.  Bound: HBM (d_out and the routed rows of src read, the
// routed rows of d_src written).  A workgroup owns a token: its slots are
// taken JB at a time, so d_out is read from HBM once and from the cache for
// each further JB slots; the dot products are summed per thread over the
// columns, then over the lanes and waves in a fixed order.
// ---------------------------------------------------------------------------
template <int T>
__global__ __launch_bounds__(kCombineThreads) void group_combine_grad_kernel(const CombineArgs a)
{
    constexpr int JB = 4, WAVES = kCombineThreads / 64;
    __shared__ float part[WAVES][JB];
    const int64_t t = blockIdx.x;
    const int w = wave_id(), l = lane_id();
    for (int j0 = 0; j0 < a.topk; j0 += JB) {
        int row[JB];
        float wt[JB], dot[JB];
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            row[j] = j0 + j < a.topk ? a.slot_row[t * a.topk + j0 + j] : -1;
            row[j] = (uint32_t)row[j] < (uint32_t)a.src_rows ? row[j] : -1;
            wt[j] = row[j] >= 0 && a.weights ? a.weights[t * a.topk + j0 + j] : 1.f;
            dot[j] = 0.f;
        }
        for (int64_t col = threadIdx.x * 8; col < a.N; col += kCombineThreads * 8) {
            float d[8];
            load8<T>(a.d_out, (size_t)t * a.N + col, d);
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                if (row[j] < 0)
                    continue;
                const size_t at = (size_t)row[j] * a.N + col;
                float v[8];
                if (a.d_weights) {
                    load8<T>(a.src, at, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dot[j] = fmaf(d[i], v[i], dot[j]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = wt[j] * d[i];
                store8<T>(a.out, at, v);
            }
        }
        if (!a.d_weights)
            continue;
#pragma unroll
        for (int j = 0; j < JB; ++j) {
#pragma unroll
            for (int m = 32; m; m >>= 1)
                dot[j] += __shfl_xor(dot[j], m);
            if (l == 0)
                part[w][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < JB && j0 + (int)threadIdx.x < a.topk) {
            float sum = 0.f;
#pragma unroll
            for (int ww = 0; ww < WAVES; ++ww)
                sum += part[ww][threadIdx.x];
            a.d_weights[t * a.topk + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

// One workgroup per token, the tokens in as many launches as their number needs
// (one up to 2^23).
hipError_t launch_group_combine_grad(const CombineArgs &args, hipStream_t s)
{
    const dim3 threads(kCombineThreads);
    const int64_t bytes = args.type == kOutF32 ? 4 : 2;
    for (int64_t first = 0; first < args.tokens; first += kCombineBlocks) {
        CombineArgs a = args;
        a.tokens = args.tokens - first < kCombineBlocks ? args.tokens - first : kCombineBlocks;
        a.d_out = (const uint8_t *)args.d_out + first * args.N * bytes;
        a.slot_row += first * args.topk;
        if (a.weights)
            a.weights += first * args.topk;
        if (a.d_weights)
            a.d_weights += first * args.topk;
        const dim3 grid((unsigned)a.tokens);
        if (a.type == kOutF32)
            hipLaunchKernelGGL(group_combine_grad_kernel<kOutF32>, grid, threads, 0, s, a);
        else
            hipLaunchKernelGGL(group_combine_grad_kernel<kOutBf16>, grid, threads, 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// ---------------------------------------------------------------------------
// d_z = d_c * act'(z) and its column sums per row group.  Bound: HBM (6 bytes
// per element in bf16).  Rows are cut into chunks that never cross a group; a
// workgroup takes one chunk and 512 columns, lane l of each of its 4 waves
// columns 8 l .. 8 l + 7, wave w the chunk's rows w, w + 4, ...  The chunk's
// column sums go to the workspace and a second, small launch adds a group's
// chunks in order: no atomics, so d_bias is the same on every run.
// ---------------------------------------------------------------------------
namespace {

constexpr int kActThreads = 256;
constexpr int kActWaves = kActThreads / 64;
constexpr int kActCols = 512;

// act'(z).  The logistic and normal factors underflow long before z = -100,
// where z times 0 would turn -inf into NaN; NaN passes through.
template <int ACT>
__device__ inline float act_slope(float z)
{
    if constexpr (ACT == kActRelu) {
        return z > 0.f ? 1.f : 0.f;
    } else if constexpr (ACT == kActSilu) {
        const float c = z < -100.f ? -100.f : (z > 100.f ? 100.f : z);
        // the hardware's exponential and reciprocal, each within an ulp or so:
        // with expf and a division the kernel was bound by its arithmetic
        // (8192 x 8192 bf16 with d_bias: 92 us; 87 so)
        const float p = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(c * -1.44269504088896340736f));
        return p * (1.f + c * (1.f - p));
    } else if constexpr (ACT == kActGelu) {
        const float c = z < -100.f ? -100.f : (z > 100.f ? 100.f : z);
        // phi's exponent on the hardware's 2^x: c^2 / 2 log2 e
        const float phi = 0.39894228040143267794f * __builtin_amdgcn_exp2f(c * c * -0.72134752044448170368f);
        return 0.5f * (1.f + erff(c * 0.70710678118654752440f)) + c * phi;
    }
    return 1.f;
}

}  // namespace

template <int T, int ACT>
__global__ __launch_bounds__(kActThreads) void act_grad_kernel(const ActGradArgs a)
{
    __shared__ float red[kActWaves][kActCols];
    const int w = wave_id(), l = lane_id();
    int r0, rows;
    if (a.offsets) {
        const GroupScan s = group_scan(a.offsets, a.groups, a.M, a.chunk);
        if ((int)blockIdx.x >= s.total)
            return;
        const GroupTile g = group_find(s, a.offsets, a.groups, a.M, a.chunk, blockIdx.x);
        r0 = g.lo + ((int)blockIdx.x - g.first) * a.chunk;
        rows = min(a.chunk, g.hi - r0);
    } else {
        r0 = blockIdx.x * a.chunk;
        rows = min(a.chunk, a.M - r0);
    }
    const int64_t col = (int64_t)blockIdx.y * kActCols + l * 8;
    float sum[8] = {};
    if (col < a.N) {
#pragma unroll 4
        for (int r = w; r < rows; r += kActWaves) {
            const size_t at = (size_t)(r0 + r) * a.N + col;
            float d[8];
            load8<T>(a.d_c, at, d);
            if constexpr (ACT != kActNone) {
                float z[8];
                load8<T>(a.z, at, z);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] *= act_slope<ACT>(z[i]);
            }
            store8<T>(a.d_z, at, d);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[i] += d[i];
        }
    }
    if (!a.partial)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        red[w][l * 8 + i] = sum[i];
    __syncthreads();
    for (int c = threadIdx.x; c < kActCols; c += kActThreads) {
        const int64_t n = (int64_t)blockIdx.y * kActCols + c;
        if (n < a.N)
            a.partial[(size_t)blockIdx.x * a.N + n] = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
    }
}

// d_bias[g][n] = the sum over the group's chunks, in order: each wave of a
// workgroup adds a quarter of them for 256 columns, then the quarters join.
__global__ __launch_bounds__(kActThreads) void act_grad_bias_kernel(const ActGradArgs a)
{
    __shared__ float red[kActWaves][256];
    const int w = wave_id(), l = lane_id();
    const int g = blockIdx.y;
    int first = 0, chunks;
    if (a.offsets) {
        const GroupScan s = group_scan(a.offsets, a.groups, a.M, a.chunk);
        const int lane = g / s.per;
        first = __builtin_amdgcn_readlane(s.excl, lane);
        for (int i = lane * s.per; i < g; ++i) {
            const int lo = group_lo(a.offsets, i, a.M);
            first += (group_hi(a.offsets, i, a.M, lo) - lo + a.chunk - 1) / a.chunk;
        }
        const int lo = group_lo(a.offsets, g, a.M);
        chunks = (group_hi(a.offsets, g, a.M, lo) - lo + a.chunk - 1) / a.chunk;
        // offsets that run backwards could count more chunks than were written
        chunks = max(0, min(chunks, a.max_chunks - first));
    } else {
        chunks = (a.M + a.chunk - 1) / a.chunk;
    }
    const int per = (chunks + kActWaves - 1) / kActWaves;
    const int c0 = min(w * per, chunks), c1 = min(c0 + per, chunks);
    const int64_t col = (int64_t)blockIdx.x * 256 + l * 4;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    if (col < a.N) {
#pragma unroll 8
        for (int c = c0; c < c1; ++c)
            sum += *(const f32x4 *)(a.partial + (size_t)(first + c) * a.N + col);
    }
    *(f32x4 *)&red[w][l * 4] = sum;
    __syncthreads();
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n < a.N)
        a.d_bias[(size_t)g * a.N + n] =
            (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
}

template <int T>
static void launch_act(const ActGradArgs &a, dim3 grid, hipStream_t s)
{
    const dim3 threads(kActThreads);
    if (a.act == kActRelu)
        hipLaunchKernelGGL((act_grad_kernel<T, kActRelu>), grid, threads, 0, s, a);
    else if (a.act == kActSilu)
        hipLaunchKernelGGL((act_grad_kernel<T, kActSilu>), grid, threads, 0, s, a);
    else if (a.act == kActGelu)
        hipLaunchKernelGGL((act_grad_kernel<T, kActGelu>), grid, threads, 0, s, a);
    else
        hipLaunchKernelGGL((act_grad_kernel<T, kActNone>), grid, threads, 0, s, a);
}

hipError_t launch_act_grad(const ActGradArgs &a, hipStream_t s)
{
    if (a.max_chunks > 0) {
        const dim3 grid((unsigned)a.max_chunks, (unsigned)((a.N + kActCols - 1) / kActCols));
        if (a.type == kOutF32)
            launch_act<kOutF32>(a, grid, s);
        else
            launch_act<kOutBf16>(a, grid, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    if (!a.d_bias)
        return hipSuccess;
    hipLaunchKernelGGL(act_grad_bias_kernel, dim3((unsigned)((a.N + 255) / 256), (unsigned)a.groups),
                       dim3(kActThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace tg
