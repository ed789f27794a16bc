// Roots and reciprocals of the AdamW kernels, from the hardware's approximations.
#pragma once

#include <float.h>

#include "types.cuh"

namespace tt {

// 1 / x (normal x) and the root of x within an ulp: of the update only, not of what an 8-bit code depends on
__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float root(float x)
{
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Minus the roots of two values, to nearest, from minus the values: signs that packed instructions cannot
// change are saved that way.  With r near 1 / sqrt(x), s = x r is near the root and s^2 - x, which the
// fused multiply-add gives exactly, is what its square is off; Heron's step s - (s^2 - x) / (2 s) =
// s - (s^2 - x) r / 2 then rounds once.  That alone leaves results next to the nearest one possible, for
// some r: with this card's, a test compares all values from 2^-102 on with the correctly rounded root.
// Below that the difference loses places.  0 gives 0, values below the least normal number a root that
// is too small, infinity NaN.
__device__ __forceinline__ F2 minus_root2(F2 minus_x)
{
    F2 r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(fmaxf(-minus_x.x, FLT_MIN)));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(fmaxf(-minus_x.y, FLT_MIN)));
    const F2 minus_s = mul2(minus_x, r);
    return fma2(fma2(minus_s, minus_s, minus_x), mul2(r, both(0.5f)), minus_s);
}

// 1 / x to nearest, without a branch, for x from 2^-100 to below 2^126, by a Newton step on an approximation r:
// 1 - x r is exact in a fused multiply-add, and r + r (1 - x r) rounds once.  As above, that r is near
// enough for every one of these values is what a test shows, not the step: for x = 2 - 2^-23 an r of
// 0.5 would give 0.5, which is not the nearest.
__device__ __forceinline__ float inverse(float x)
{
    const float r = rcp(x);
    return __fmaf_rn(__fmaf_rn(-x, r, 1.f), r, r);
}

}  // namespace tt
