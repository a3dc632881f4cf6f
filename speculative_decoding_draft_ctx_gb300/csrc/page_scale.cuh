// Codes of page-scaled caches: e4m3 values times a power of two per page and
// head.  Re-encoding to a larger power of two divides the code by a power of two,
// which is exact in fp16 down to its last bit, 2^-24 (what lies below ends below
// half the smallest code, 2^-10, and becomes zero either way), then rounds once.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "draft_step_internal.h"

namespace dspark {

// a page's exponent, kept to its range
__device__ __forceinline__ int page_exponent(const int8_t *scales, int64_t page, int heads, int h, int part)
{
    const int e = scales[(page * heads + h) * 2 + part];
    return min(max(e, kScaleMin), kScaleMax);
}

// 2^-d as an fp16 pair (0 from d = 25 on: a code times it is below 2^-16)
__device__ __forceinline__ uint32_t half2_power(int d)
{
    const uint32_t h = d <= 14 ? (uint32_t)(15 - d) << 10 : d <= 24 ? 1u << (24 - d) : 0u;
    return h * 0x10001u;
}

// four codes times the fp16 pair f
__device__ __forceinline__ uint32_t scale_codes(uint32_t w, uint32_t f)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 a, b;\n\t"
        "mov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 a, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 b, hi;\n\t"
        "mul.rn.f16x2 a, a, %2;\n\t"
        "mul.rn.f16x2 b, b, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 lo, a;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 hi, b;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "r"(w), "r"(f));
    return r;
}

__device__ __forceinline__ uint4 scale_codes(uint4 w, uint32_t f)
{
    return make_uint4(scale_codes(w.x, f), scale_codes(w.y, f), scale_codes(w.z, f), scale_codes(w.w, f));
}

}  // namespace dspark
