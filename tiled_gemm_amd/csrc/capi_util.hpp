// What the C entry points share: the per-thread error text, argument checks
// and the device check (defined in capi.cpp).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "tgemm.h"
#include "kernels.hpp"

namespace tg {

int capi_fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int capi_ok();
int capi_check_device();
int capi_epilogue(const gemm_epilogue_args *epi, EpiArgs *out);

inline bool capi_aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool capi_overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && na && nb && x < y + nb && y < x + na;
}

}  // namespace tg
