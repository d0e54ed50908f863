// Eight consecutive columns of a row, as the memory-bound kernels move them:
// bf16 or fp32 rows to fp32 and back, and the 8-bit checkpoint's elements.
#pragma once

#include "device.hpp"

namespace tg {

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

// ---------------------------------------------------------------------------
// The 8-bit checkpoint: e4m3 elements, one E8M0 scale (2^(byte - 127); 255 is
// NaN) per kCkptBlock consecutive columns of a row.
// ---------------------------------------------------------------------------
constexpr int kCkptBlock = 32;

typedef float f32x2_t __attribute__((ext_vector_type(2)));

__device__ inline float e8m0_value(uint32_t byte)
{
    return byte == 255u ? __builtin_nanf("") : (byte == 0u ? as_f32(0x00400000u) : as_f32(byte << 23));
}

// Eight elements (8-byte aligned) times their block's scale.  The product of
// a 4-bit significand and a power of two is exact in fp32 unless it leaves
// fp32's range.
__device__ inline void ckpt_load8(const uint8_t *q, size_t at, float step, float (&v)[8])
{
    const u32x2 w = *(const u32x2 *)(q + at);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
        const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
        v[4 * h] = lo.x * step;
        v[4 * h + 1] = lo.y * step;
        v[4 * h + 2] = hi.x * step;
        v[4 * h + 3] = hi.y * step;
    }
}

}  // namespace tg
