// One row of values to the library's FP8 storage: E4M3FN codes and one fp32
// scale, scale = max|x| / 448 (1 for an all-zero row), code = the E4M3FN value
// nearest to the correctly rounded quotient x / scale, ties to even.
//
// An infinite element makes the scale infinite and is stored as +-448, its own
// sign: it reads as itself (and the row's finite elements, codes 0, as NaN).  A
// zero whose row's scale underflows to 0 stays a zero.  A NaN does not enter
// the scale; KEEP_NAN stores it as a NaN code, else it takes a finite one.
#pragma once

#include "common.h"

namespace dsaidx {

constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float row_scale(float absmax) { return absmax > 0.f ? absmax / kE4m3Max : 1.f; }

// Codes of eight consecutive elements of a row with this scale.
template <bool KEEP_NAN>
__device__ __forceinline__ uint2 quant8(const float (&x)[8], float scale) {
    float q[8];
    if (scale >= 0x1p-80f && scale <= 0x1p+80f) {
        // RN(x / scale) from y = RN(1 / scale) (one correctly rounded
        // division per row): q0 = RN(x y) lies within 1.5 ulp of
        // x / scale; one correction q1 = RN(q0 + r0 y) with the
        // remainder r0 = x - scale q0 taken in an fma is within half an
        // ulp plus a few 2^-24 ulp, so faithful; the remainder of a
        // faithful quotient is exact, and one more correction from it
        // gives the correctly rounded quotient (Markstein's theorem for
        // a correctly rounded reciprocal).  No step overflows (|x y| <=
        // 448.1) and the remainders stay off the subnormal grid for
        // |x| >= 2^-100; below that the quotient is under 2^-19, whose
        // E4M3 code is a signed zero on any path.  The sign is put back
        // for x = -0, which the corrections turn into +0.
        const float y = 1.f / scale;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q0 = x[j] * y;
            const float q1 = fmaf(fmaf(-scale, q0, x[j]), y, q0);
            const float q2 = fmaf(fmaf(-scale, q1, x[j]), y, q1);
            q[j] = __builtin_copysignf(q2, x[j]);
            // |x| <= 448 scale (1 + 2^-24): the quotient is below the midpoint above
            // 448 in any case, and the clamp only there for NaN
            if constexpr (!KEEP_NAN) q[j] = fminf(fmaxf(q[j], -kE4m3Max), kE4m3Max);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float r = x[j] / scale;   // NaN: inf / inf, 0 / 0 or x itself
            q[j] = r == r ? fminf(fmaxf(r, -kE4m3Max), kE4m3Max)
                          : __builtin_copysignf(x[j] == 0.f ? 0.f : kE4m3Max, x[j]);
            if constexpr (KEEP_NAN) q[j] = x[j] == x[j] ? q[j] : x[j];
        }
    }
    int w0 = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    w0 = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w0, true);
    int w1 = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    w1 = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], w1, true);
    return uint2{(uint32_t)w0, (uint32_t)w1};
}

}  // namespace dsaidx
