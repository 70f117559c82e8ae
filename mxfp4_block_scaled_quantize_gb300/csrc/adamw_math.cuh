// adamw_math.cuh -- the roots and quotients of the 8-bit moments, from a few operations without a
// branch each: a residual computed exactly by a fused multiply-add corrects an approximate result
// to the correctly rounded one (P. Markstein, IBM J. Res. Dev. 34, 1990).  Both are compared with
// CUDA's rounded intrinsics by the GPU tests, the root for every float.
#pragma once

#include <cstdint>

namespace mxfp4 {

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// x / s from inv = the correctly rounded 1 / s, for |x| <= 448 s (1 + 2^-22): q = x inv and the exact
// residual x - q s give the quotient as q + residual inv.  Equal to __fdiv_rn(x, s) for |x| >=
// 2^-100.  Below, the residual loses bits to the end of fp32's range, and the result is within 2 ulp.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
    const float q = __fmul_rn(x, inv);
    return __fmaf_rn(__fmaf_rn(-q, s, x), inv, q);
}

// Square roots of eight values >= 0: y = 1 / sqrt(v) approximately, s = v y, and one correction
// by the exact residual, s + (v - s^2) y / 2 (Markstein, as above), without a branch an element.
// Equal to __fsqrt_rn for every float from 0 to infinity.  Values outside [2^-100, 2^126), where a
// residual could lose bits, zero among them, take __fsqrt_rn.
__device__ __forceinline__ void sqrt8(const float* v, float* r) {
    float lo = v[0], hi = v[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) {
        lo = fminf(lo, v[k]);
        hi = max_nan(hi, v[k]);
    }
    if (lo >= 7.8886091e-31f && hi < 8.5070592e37f) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float y;
            asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v[k]));
            const float s = __fmul_rn(v[k], y);
            r[k] = __fmaf_rn(__fmaf_rn(-s, s, v[k]), 0.5f * y, s);
        }
    } else {
#pragma unroll 1
        for (int k = 0; k < 8; ++k) r[k] = __fsqrt_rn(v[k]);
    }
}

}  // namespace mxfp4
