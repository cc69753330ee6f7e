// fd_e4m3.cuh -- float32 values divided by a scale and rounded to E4M3 bytes,
// for the kernels that write an E4M3 cache.
#pragma once

#include <stdint.h>

namespace fd {

// Two floats to two E4M3 bytes (the first in the lower), to nearest, ties to
// even, saturated; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    return e4m3x2(a, b) | e4m3x2(c, d) << 16;
}

// The bytes of f[i] / scale (IEEE division), four a word.
// The quotient lies between the products with a reciprocal that is a little
// too small and one that is a little too large (2^-21, against 3 roundings of
// 2^-24), and rounding keeps that order: where both give the same byte, it is
// the quotient's.  Else (ties, one in 10^5 otherwise, and scales whose
// reciprocal is no normal number) divide.
template <int EL> __device__ __forceinline__ void e4m3_quotients(const float *f, float scale, uint32_t (&w)[EL / 4])
{
    const float r = __frcp_rn(scale);
    const float r0 = r * (1.f - 0x1p-21f), r1 = r * (1.f + 0x1p-21f);
    bool same = fabsf(scale) >= 0x1p-126f && fabsf(scale) <= 0x1p125f;
#pragma unroll
    for (int k = 0; k < EL / 4; ++k) {
        w[k] = e4m3x4(f[4 * k] * r0, f[4 * k + 1] * r0, f[4 * k + 2] * r0, f[4 * k + 3] * r0);
        same &= w[k] == e4m3x4(f[4 * k] * r1, f[4 * k + 1] * r1, f[4 * k + 2] * r1, f[4 * k + 3] * r1);
    }
    if (!same) {
#pragma unroll
        for (int k = 0; k < EL / 4; ++k)
            w[k] = e4m3x4(__fdiv_rn(f[4 * k], scale), __fdiv_rn(f[4 * k + 1], scale), __fdiv_rn(f[4 * k + 2], scale),
                          __fdiv_rn(f[4 * k + 3], scale));
    }
}

}  // namespace fd
