// Low-rank adapters of many requests, the first half:
//
//   v[m][r] / s_a = sum_k x[m][k] down_a[r][k],     a the adapter of row m
//
// for the projection's kernel to finish (lora.hpp), which also scales: fp32 sums
// over parts of K.
//
// A CU alone streams some 30 to 50 GB/s, so what counts is the bytes that each
// workgroup reads and that there are enough workgroups: K is cut into parts (up
// to kLoraParts), which the reader adds.  Two forms, by the number of rows:
//   * up to kFewRows (decode): the adapters' matrices are the bytes, most rows
//     have one of their own.  A workgroup takes one adapter of 16 rows, 16 of its
//     ranks and one part.  (200 rows, K 4160, rank 64: 11.5 us in packed prompts,
//     18.7 with 16 adapters in random order; the other form 10.8 and 29.6.  600
//     rows: 21.0 packed against 12.4.)
//   * above (prompts, training): x is the bytes, and blocks of rows mostly have
//     one adapter.  A workgroup takes the first adapter of 16, 32 or 64 rows (so
//     many that the parts still give every CU one) with up to 64 ranks at once,
//     x read once for them.  The further adapters of a block (decode rows in
//     front of the prompts, a prompt's end) are shared out to some workgroups
//     more (more_of), which read the rows of theirs only.  One after the other in
//     the block's own workgroup, 16 of them took 260 us (4001 x 4160, rank 64).  As it
//     is 18 us for 42 MB with them, 14.8 us for 34 MB with one adapter: 2.3 TB/s, a
//     few steps of K per wave, so mostly latency.  Rows in random order, where
//     every block has all adapters, are what this form is not made for: both
//     halves for 1000 / 3000 x 4096 x 4160, rank 64, 16 adapters 193 / 507 us, packed
//     81 / 139; 8192 x 4096 x 4096, rank 16, 64 adapters 1783, packed 255.
#include "lora.hpp"
#include "stream.hpp"

namespace tg {

namespace {

constexpr int kFewRows = 256;
// Workgroups for the further adapters of all blocks: many beside small blocks, few
// beside those of 64 rows, which fill the CUs with one round of workgroups (see
// lora_down_many_kernel).
constexpr int more_of(int rows) { return rows == 64 ? 16 : 64; }
constexpr int kWindow = 512;              // groups of 64 rows that they look through at a time
constexpr int kStepBytes = 64;            // of K, per row (stream.hpp)

int more_wgs(int adapters, int rows) { return adapters > 1 ? more_of(rows) : 0; }

// Rows of a workgroup's block in the form for many rows.  Measured, 16 / 32 / 64 in
// us (K 4160, rank 64): one adapter, 1000 rows 7.3 / 8.3 / 10.9, 1500 rows 11.7 / 9.0 /
// 11.1, 3000 rows 21.1 / 15.2 / 12.8; packed prompts of 16 adapters, 2000 rows 21 / 16 /
// 14, 4000 rows 32 / 30 / 18.
int many_rows(int64_t M) { return M <= 1024 ? 16 : M <= 2048 ? 32 : 64; }

// The n-th adapter (in the order of its first row) among the rows of `mask`, or
// -1; same: its rows.  id: one row per lane, -1 without an adapter.  (The result
// is the same in every lane; saying so keeps the loads behind it from being
// issued lane value by lane value.)
__device__ inline int lora_nth(int id, unsigned long long mask, int n, unsigned long long *same)
{
    unsigned long long left = __ballot(id >= 0) & mask;
    int e = -1;
    while (left) {
        const int at = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const unsigned long long rows = __ballot(id == at) & mask;
        left &= ~rows;
        if (n-- == 0) {
            e = at;
            *same = rows;
            break;
        }
    }
    return __builtin_amdgcn_readfirstlane(e);
}

// The product of the 16 MB rows from m0 on (those of `there`, bit r: row m0 + r)
// with an adapter, ranks 16 NB rb .., K steps of part `part`.  find(same) names the
// adapter (-1: none, nothing is stored) and the rows that are stored; it is called
// behind the first loads of x.
template <int MB, int NB, typename FindAdapter>
__device__ inline void lora_down(const LoraArgs &a, int m0, unsigned long long there, FindAdapter find_adapter, int rb,
                                 int part, float (*red)[16 * MB][stream_pitch<NB>()])
{
    const int r16 = lane_id() & 15;
    const uint32_t kb = (uint32_t)a.K * 2u;
    const int steps = (int)(kb / 64), per = (steps + a.parts - 1) / a.parts;
    const int step0 = min(part * per, steps), n_steps = min(per, steps - step0);
    const auto rX = make_rsrc((const uint8_t *)a.x + (size_t)m0 * kb, (uint32_t)min(a.M - m0, 16 * MB) * kb);
    uint32_t xoff[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i)                     // (rows past M are past the record count)
        xoff[i] = keep_or_oob((there >> (i * 16 + r16)) & 1, (uint32_t)(i * 16 + r16) * kb);
    unsigned long long same = 0;
    auto find = [&](__amdgpu_buffer_rsrc_t (&rB)[NB]) {
        const int e = find_adapter(&same), any = e < 0 ? 0 : e;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            // ranks past the last (of a padded block) read zeros
            const int r = min((rb * NB + j) * 16, a.rank);
            const uint32_t bytes = e < 0 ? 0u : (uint32_t)(a.rank - r < 16 ? a.rank - r : 16) * kb;
            rB[j] = make_rsrc((const uint8_t *)a.down + ((size_t)any * a.rank + r) * kb,
                              (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes));
        }
    };
    // (Steps per set of loads, one block of ranks and more: with 2 instead of 1 for
    // more, 4001 x 4160 and rank 64 in packed prompts takes 30.3 instead of 29.5 us,
    // 8192 x 2048 and rank 32 19.0 instead of 16.7.)
    stream_product<MB, NB, false, false, NB == 1 ? 4 : 1>(rX, xoff, find, kb, step0, n_steps, red);
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * MB * 16 * NB; o += kStreamThreads) {
        const int row = o / (16 * NB), col = o % (16 * NB), r = rb * 16 * NB + col;
        if (!((same >> row) & 1) || r >= a.rank)
            continue;
        a.v[((size_t)part * a.M + m0 + row) * a.rank_pad + r] = stream_sum<MB, NB>(red, row, col);
    }
}

}  // namespace

__global__ __launch_bounds__(kStreamThreads, 4) void lora_down_few_kernel(const LoraArgs a)
{
    __shared__ float red[kStreamWaves][16][stream_pitch<1>()];
    const int m0 = blockIdx.x * 16, l = lane_id();
    const int rb = blockIdx.z / a.parts, part = blockIdx.z - rb * a.parts;
    unsigned long long same = 0;
    const int e = lora_nth(lora_id(a, l < 16 && m0 + l < a.M, m0 + l), ~0ull, blockIdx.y, &same);
    if (e < 0)                                       // (most workgroups, where rows share adapters)
        return;
    auto find = [&](unsigned long long *rows) {
        *rows = same;
        return e;
    };
    lora_down<1, 1>(a, m0, same, find, rb, part, red);
}

// Adapters beyond the first in each of the 4 / MB blocks of 64 rows, together.
template <int MB>
__device__ inline int lora_further(int id)
{
    int n = 0;
#pragma unroll
    for (int b = 0; b < 4 / MB; ++b) {
        unsigned long long left = __ballot(id >= 0) & ((~0ull >> (64 - 16 * MB)) << (16 * MB * b));
        for (bool first = true; left; first = false) {
            left &= ~__ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctzll(left)));
            n += !first;
        }
    }
    return __builtin_amdgcn_readfirstlane(n);
}

// Workgroups more ..: the first adapter of each block of 16 MB rows.  The `more`
// (0 or kMore) before them: each looks through all rows' adapters for the
// blocks that have more than one and takes every kMore-th of what it finds.
// (Before, so that what they find is not left to the end.)  4001 x 4160, rank 64,
// 16 decode rows and 6 prompts of up to 16 adapters: 18.5 us with 16 of them (and
// three parts), 30 with 32, a second round of workgroups, 27 with 8; with one
// adapter 14.8.  Blocks of 16 rows: 64 take 12.4 us for 600 packed rows and 113
// for 1000 rows with 16 adapters in random order, 16 take 11.3 and 216.
template <int MB, int NB>
__global__ __launch_bounds__(kStreamThreads, 2) void lora_down_many_kernel(const LoraArgs a, int more)
{
    __shared__ float red[kStreamWaves][16 * MB][stream_pitch<NB>()];
    __shared__ int32_t count[kWindow];
    constexpr int kMore = more_of(16 * MB);
    static_assert((kMore & (kMore - 1)) == 0, "a power of two");
    const int l = lane_id(), rb = blockIdx.y, part = blockIdx.z;
    if ((int)blockIdx.x >= more) {
        const int m0 = ((int)blockIdx.x - more) * 16 * MB;
        const int id = lora_id(a, l < 16 * MB && m0 + l < a.M, m0 + l);
        auto find = [&](unsigned long long *rows) { return lora_nth(id, ~0ull, 0, rows); };
        lora_down<MB, NB>(a, m0, ~0ull, find, rb, part, red);
        return;
    }
    const int mine = blockIdx.x, groups = (a.M + 63) / 64;
    int k = 0;                                       // adapters found so far
    for (int g0 = 0; g0 < groups; g0 += kWindow) {
        const int here = min(groups - g0, kWindow);
        __syncthreads();
        for (int i = wave_id() * 8; i < here; i += kStreamWaves * 8) {
            int id[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {            // in flight together
                const int row = (g0 + i + u) * 64 + l;
                id[u] = lora_id(a, row < a.M, row);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int n = lora_further<MB>(id[u]);
                if (l == 0 && i + u < here)
                    count[i + u] = n;
            }
        }
        __syncthreads();
        for (int i = 0; i < here; i += 64) {
            const int n = i + l < here ? count[i + l] : 0;
            for (unsigned long long some = __ballot(n > 0); some; some &= some - 1) {
                const int at = __builtin_ctzll(some), g = g0 + i + at;
                const int last = k + __builtin_amdgcn_readlane(n, at);
                if (k + ((mine - k) & (kMore - 1)) >= last) {       // none of these is this workgroup's
                    k = last;
                    continue;
                }
                const int id = lora_id(a, g * 64 + l < a.M, g * 64 + l);
                for (int b = 0; b < 4 / MB; ++b) {
                    const unsigned long long mask = (~0ull >> (64 - 16 * MB)) << (16 * MB * b);
                    unsigned long long left = __ballot(id >= 0) & mask;
                    for (bool first = true; left; first = false) {
                        // (the same in every lane, see lora_nth)
                        const int e = __builtin_amdgcn_readfirstlane(
                            __builtin_amdgcn_readlane(id, __builtin_ctzll(left)));
                        const unsigned long long same = __ballot(id == e) & mask;
                        left &= ~same;
                        if (first || (k++ & (kMore - 1)) != mine)
                            continue;
                        auto find = [&](unsigned long long *rows) {
                            *rows = same >> (16 * MB * b);
                            return e;
                        };
                        lora_down<MB, NB>(a, g * 64 + 16 * MB * b, same >> (16 * MB * b), find, rb, part, red);
                        __syncthreads();
                    }
                }
            }
        }
    }
}

namespace {

template <int MB, int NB>
hipError_t many(const LoraArgs &a, int passes, hipStream_t s)
{
    const int64_t blocks = ((int64_t)a.M + 16 * MB - 1) / (16 * MB);
    const int more = more_wgs(a.adapters, 16 * MB);
    hipLaunchKernelGGL((lora_down_many_kernel<MB, NB>),
                       dim3((unsigned)(blocks + more), (unsigned)passes, (unsigned)a.parts), dim3(kStreamThreads), 0, s,
                       a, more);
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

// Parts of K, never less than a step of K per wave.  Few rows: 64 KiB of 16 ranks
// each.  Many: as many as bring the launch's rounds of workgroups nearest to full
// (fewest rounds over parts; the LDS of 64 rows by 64 ranks leaves one workgroup
// per CU, that of 16 or 32 rows two or more).  4001 x 4160 and rank 64 in packed
// prompts: 22.3 us with the 3 parts that make one round of them, 24.6 with 4;
// 8000 x 4160 with one adapter 28.3 with 2, 31.0 with 4.  64 rows by 32 ranks leave
// two workgroups per CU, but counted as one they take as long or less, as the tiles
// read every part: 8192 x 8192 x 2048 one adapter 308 us in all with 2 parts, 315 with 4;
// 4096 x 4096 x 4096 packed 134 / 138, 6000 x 2048 x 2048 73 / 75, 8192 x 4096 x 4096 250 / 249,
// 3000 x 8192 x 8192 382 / 382.
int lora_parts(int64_t M, int64_t K, int rank_pad, int adapters)
{
    const int64_t most = K * 2 / kStepBytes / kStreamWaves;
    const int64_t cap = most < 1 ? 1 : most > kLoraParts ? kLoraParts : most;
    if (M <= kFewRows) {
        const int64_t p = (K * 2 * 16 + (64 << 10) - 1) / (64 << 10);
        return (int)(p < 1 ? 1 : p > cap ? cap : p);
    }
    const int64_t rows = many_rows(M), passes = rank_pad == 32 ? 1 : (rank_pad + 63) / 64;
    const int64_t wgs = ((M + rows - 1) / rows + more_wgs(adapters, (int)rows)) * passes;
    const int64_t slots = rows == 64 ? 256 : 512;
    int64_t best = 1, best_rounds = 0;
    for (int64_t p = 1; p <= cap; ++p) {
        const int64_t rounds = (wgs * p + slots - 1) / slots;
        if (p == 1 || rounds * best < best_rounds * p) {
            best = p;
            best_rounds = rounds;
        }
    }
    return (int)best;
}

hipError_t launch_lora_down(const LoraArgs &a, hipStream_t s)
{
    const int blocks = a.rank_pad / 16;
    if (a.M <= kFewRows) {
        const unsigned rows = (unsigned)((a.M + 15) / 16);
        hipLaunchKernelGGL(lora_down_few_kernel,
                           dim3(rows, (unsigned)(a.adapters < 16 ? a.adapters : 16), (unsigned)(blocks * a.parts)),
                           dim3(kStreamThreads), 0, s, a);
        return hipGetLastError();
    }
    const int rows = many_rows(a.M);
    return rows == 16 ? many_mb<1>(a, blocks, s) : rows == 32 ? many_mb<2>(a, blocks, s) : many_mb<4>(a, blocks, s);
}

}  // namespace tg
