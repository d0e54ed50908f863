// Activations kept in 8 bits between the forward and the backward pass: every
// 32 columns of a row become 32 e4m3 elements and one power of two,
//
//   s = the smallest power of two with  max |x| <= 448 s  over the block's finite x
//   q = e4m3(x / s),   value = q s
//
// 448 being e4m3's largest number: the division is exact, so each element is
// rounded once (to nearest even, at most 2^-4 of itself while it stays above
// 2^-6 s), and none is clipped.  The pair (q, exponent byte) is the MX form
// that the MXFP8 products read.
//
// Both kernels are bound by HBM: pack reads 2 (bf16) or 4 bytes and writes
// 33 / 32 per element, unpack the other way round.  8192 x 8192 bf16 packed in 37 us,
// 5.5 TB/s; 8192 x 4096 unpacked with SiLU in 20 us, 5.0 TB/s.  A wave takes 512 columns of
// kPackRows rows, a lane 8 consecutive columns of each (16-byte loads), so 4
// lanes hold a block and find its largest magnitude with two lane moves.
#include "cols.hpp"

namespace tg {

namespace {

constexpr int kCkptThreads = 256;
constexpr int kCkptWaves = kCkptThreads / 64;
constexpr int kCkptCols = 512;
// Rows per wave: their loads are in flight together.  Measured, 1 / 2 / 4 / 8 rows in
// us: pack 8192 x 8192 bf16 39.1 / 36.9 / 40.3 / 42.7; unpack 8192 x 4096 with SiLU
// 2 / 3 / 4 / 8: 22.5 / 21.9 / 21.4 / 22.6.
constexpr int kPackRows = 2, kUnpackRows = 4;
// A launch has fewer than 2^32 threads.
constexpr int64_t kCkptBlocks = (int64_t)1 << 23;

// (GELU: normal_cdf's error shows in fp32 only; see there.)
template <int T, int ACT>
__device__ inline float ckpt_act(float z)
{
    float e;
    return ACT == kActSilu ? epi_silu(z) : ACT == kActGelu && T == kOutBf16 ? z * normal_cdf(z, e) : epi_act(z, ACT);
}

// The largest of the 4 lanes' values that share a block.
__device__ inline uint32_t quad_max(uint32_t x)
{
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true));     // lanes 1 0 3 2
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

// A wave's place: 512 columns of ROWS rows; `col` is this lane's first column.
struct CkptPlace {
    int64_t row, col;
};
template <int ROWS>
__device__ inline CkptPlace ckpt_place(uint32_t unit, uint32_t chunks)
{
    const uint32_t r = unit / chunks;
    return CkptPlace{(int64_t)r * ROWS, (int64_t)(unit - r * chunks) * kCkptCols + lane_id() * 8};
}

}  // namespace

template <int T>
__global__ __launch_bounds__(kCkptThreads) void ckpt_pack_kernel(const CkptArgs a)
{
    const uint32_t step = gridDim.x * kCkptWaves;
    for (uint32_t u = __builtin_amdgcn_readfirstlane(blockIdx.x * kCkptWaves + wave_id()); u < a.units; u += step) {
        const CkptPlace p = ckpt_place<kPackRows>(u, a.chunks);
        const bool in = p.col < a.N;
        float v[kPackRows][8];
#pragma unroll
        for (int r = 0; r < kPackRows; ++r) {
            if (in && p.row + r < a.M) {
                load8<T>(a.src, (size_t)(p.row + r) * a.N + p.col, v[r]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[r][i] = 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < kPackRows; ++r) {
            // Magnitudes compare as their bits.
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top = max(top, __builtin_bit_cast(uint32_t, v[r][i]) & 0x7FFFFFFFu);
            if (__ballot(top >= 0x7F800000u)) {
                // e4m3 has no infinity: it is stored as NaN, like NaN itself,
                // and neither counts for the block's scale
                top = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t m = __builtin_bit_cast(uint32_t, v[r][i]) & 0x7FFFFFFFu;
                    top = max(top, m < 0x7F800000u ? m : 0u);
                    v[r][i] = m < 0x7F800000u ? v[r][i] : as_f32(0x7FC00000u);
                }
            }
            top = quad_max(top);
            // top = 1.f 2^(e - 127); 448 = 1.75 2^8
            const int byte = max((int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), 0);
            const float inv = as_f32((uint32_t)(254 - byte) << 23);
            uint32_t w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float *x = v[r] + 4 * h;
                const int t = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, 0, false);
                w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, t, true);
            }
            if (in && p.row + r < a.M) {
                *(u32x2 *)(a.q + (size_t)(p.row + r) * a.N + p.col) = u32x2{w[0], w[1]};
                if ((lane_id() & 3) == 0)
                    a.scales[(size_t)(p.row + r) * a.blocks + p.col / kCkptBlock] = (uint8_t)byte;
            }
        }
    }
}

template <int T, int ACT>
__global__ __launch_bounds__(kCkptThreads) void ckpt_unpack_kernel(const CkptArgs a)
{
    const uint32_t step = gridDim.x * kCkptWaves;
    for (uint32_t u = __builtin_amdgcn_readfirstlane(blockIdx.x * kCkptWaves + wave_id()); u < a.units; u += step) {
        const CkptPlace p = ckpt_place<kUnpackRows>(u, a.chunks);
        if (p.col >= a.N)
            continue;
        u32x2 w[kUnpackRows];
        uint32_t byte[kUnpackRows];
#pragma unroll
        for (int r = 0; r < kUnpackRows; ++r) {        // (past the last row: that row again)
            const int64_t row = min(p.row + r, a.M - 1);
            w[r] = *(const u32x2 *)(a.q + (size_t)row * a.N + p.col);
            byte[r] = a.scales[(size_t)row * a.blocks + p.col / kCkptBlock];
        }
#pragma unroll
        for (int r = 0; r < kUnpackRows; ++r) {
            float v[8];
            ckpt_value8(w[r], e8m0_value(byte[r]), v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = ckpt_act<T, ACT>(v[i]);
            if (p.row + r < a.M)
                store8<T>(a.out, (size_t)(p.row + r) * a.N + p.col, v);
        }
    }
}

namespace {

dim3 ckpt_grid(const CkptArgs &a)
{
    const int64_t blocks = ((int64_t)a.units + kCkptWaves - 1) / kCkptWaves;
    return dim3((unsigned)(blocks < kCkptBlocks ? blocks : kCkptBlocks));
}

template <int T>
void unpack(const CkptArgs &a, hipStream_t s)
{
    const dim3 grid = ckpt_grid(a), threads(kCkptThreads);
    if (a.act == kActRelu)
        hipLaunchKernelGGL((ckpt_unpack_kernel<T, kActRelu>), grid, threads, 0, s, a);
    else if (a.act == kActSilu)
        hipLaunchKernelGGL((ckpt_unpack_kernel<T, kActSilu>), grid, threads, 0, s, a);
    else if (a.act == kActGelu)
        hipLaunchKernelGGL((ckpt_unpack_kernel<T, kActGelu>), grid, threads, 0, s, a);
    else
        hipLaunchKernelGGL((ckpt_unpack_kernel<T, kActNone>), grid, threads, 0, s, a);
}

}  // namespace

namespace {

int64_t units(int64_t M, int64_t N, int rows) { return (M + rows - 1) / rows * ((N + kCkptCols - 1) / kCkptCols); }

}  // namespace

int64_t ckpt_units(int64_t M, int64_t N) { return units(M, N, kPackRows < kUnpackRows ? kPackRows : kUnpackRows); }

hipError_t launch_ckpt_pack(const CkptArgs &args, hipStream_t s)
{
    CkptArgs a = args;
    a.chunks = (uint32_t)((a.N + kCkptCols - 1) / kCkptCols);
    a.units = (uint32_t)units(a.M, a.N, kPackRows);
    if (a.type == kOutF32)
        hipLaunchKernelGGL(ckpt_pack_kernel<kOutF32>, ckpt_grid(a), dim3(kCkptThreads), 0, s, a);
    else
        hipLaunchKernelGGL(ckpt_pack_kernel<kOutBf16>, ckpt_grid(a), dim3(kCkptThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_ckpt_unpack(const CkptArgs &args, hipStream_t s)
{
    CkptArgs a = args;
    a.chunks = (uint32_t)((a.N + kCkptCols - 1) / kCkptCols);
    a.units = (uint32_t)units(a.M, a.N, kUnpackRows);
    if (a.type == kOutF32)
        unpack<kOutF32>(a, s);
    else
        unpack<kOutBf16>(a, s);
    return hipGetLastError();
}

}  // namespace tg
