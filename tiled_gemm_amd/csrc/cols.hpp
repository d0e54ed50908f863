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

// Two fp32 -> two bf16 (nearest even) in one instruction, packed low-first: the bits
// of pack_bf16x2, which converts them one by one and joins them.
__device__ inline uint32_t pack_pair(float lo, float hi)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

template <int T>
__device__ inline void store8(void *base, size_t at, const float (&v)[8])
{
    if constexpr (T == kOutF32) {
        *(f32x4 *)((float *)base + at) = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4 *)((float *)base + at + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        *(u32x4 *)((uint16_t *)base + at) = u32x4{pack_pair(v[0], v[1]), pack_pair(v[2], v[3]),
                                                  pack_pair(v[4], v[5]), pack_pair(v[6], v[7])};
    }
}

// ---------------------------------------------------------------------------
// The 8-bit checkpoint: e4m3 elements, one E8M0 scale (2^(byte - 127); 255 is
// NaN) per kCkptBlock consecutive columns of a row.
// ---------------------------------------------------------------------------
constexpr int kCkptBlock = 32;

typedef float f32x2_t __attribute__((ext_vector_type(2)));

// 2^(byte - 127): the exponent in place, except that 0 is 2^-127, a fraction bit,
// which also makes a NaN of 255.
__device__ inline float e8m0_value(uint32_t byte)
{
    return as_f32(byte << 23 | (((byte + 1) & 0xFF) < 2 ? 0x00400000u : 0u));
}

// Eight elements times their block's scale.  The product of a 4-bit significand
// and a power of two is exact in fp32 unless it leaves fp32's range.
__device__ inline void ckpt_value8(u32x2 w, float step, float (&v)[8])
{
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

// Phi(z) and e = exp(-z^2 / 2), for GELU in bf16 beside the checkpoint's few bytes,
// where erff (two branches of long polynomials) bounded the kernels: Abramowitz and
// Stegun, 7.1.26, erfc(x) = (a1 t + .. + a5 t^5) exp(-x^2), t = 1 / (1 + p x), for
// x = |z| / sqrt 2 >= 0, within 1.5e-7 by itself.  In fp32 the coefficients of both
// signs add their rounding: Phi is within 2^-21 (2.9e-7 where t is near 1, with the
// exponential and the reciprocal rounded correctly; 2^-22.3 at most measured over
// every e4m3 number times a power of two, the slope's other term included).  That
// is absolute; of Phi itself it is 5e-4 at z = -4 and 2e-3 at -5, half a step of
// bf16, and 1% at -8.  fp32 results take erff (2^-23.7), whose time the wider rows
// mostly hide: 4096 x 4096 unpacked in 18.0 us, 17.1 so; the gradient of 4096 x 8192
// 72.6, 70.0; of 1013 x 2112 in 16 groups 14.1, 12.1.  NaN passes through.
__device__ inline float normal_cdf(float z, float &e)
{
    e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170368f);
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.3275911f * 0.70710678118654752440f, 1.f));
    float y = fmaf(t, 1.061405429f, -1.453152027f);
    y = fmaf(t, y, 1.421413741f);
    y = fmaf(t, y, -0.284496736f);
    y = fmaf(t, y, 0.254829592f);
    y = 0.5f * t * y * e;
    return z < 0.f ? y : 1.f - y;
}

}  // namespace tg
