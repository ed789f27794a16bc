// The table as a matrix: activations, what is done to a sum of products, and the kernels' arguments.
#pragma once

#include "roots.cuh"

namespace tt {

inline bool activation_known(int a) { return a >= TT_ACT_NONE && a <= TT_ACT_SOFTCAP; }

// Phi(-|z|), the normal distribution function's tail, and e = exp(-z^2 / 2), which gelu's slope needs too.  With x = |z| / sqrt(2),
// Phi(-|z|) = e erfcx(x) / 2, and erfcx(x) = exp(x^2) erfc(x) falls smoothly from 1 like 1 / x: a polynomial of t = 1 / (1 + 0.4 x)
// without a constant term, fitted to the least relative error, is within 1.4e-7 of it for all x >= 0.  What z^2 / 2 loses in its
// rounding is put back, so that the tail is right in relative terms: Phi is off by 5 steps of 2^-23 at most.
__device__ __forceinline__ float normal_tail(float z, float& e)
{
    const float w = fminf(fabsf(z), 40.f), h = -0.5f * w, a = h * w;
    e = expf(a);
    e = fmaf(e, fmaf(h, w, -a), e);
    const float t = rcp(fmaf(0.4f * 0.70710678f, fabsf(z), 1.f));
    float p = 0.050265081f;
    p = fmaf(p, t, -0.18291025f);
    p = fmaf(p, t, 0.16909297f);
    p = fmaf(p, t, -0.0056056734f);
    p = fmaf(p, t, 0.14142445f);
    p = fmaf(p, t, 0.16854656f);
    p = fmaf(p, t, 0.20784137f);
    p = fmaf(p, t, 0.22566977f);
    p = fmaf(p, t, 0.22567585f);
    return 0.5f * e * (p * t);
}

// act(z).  A z below -1e30 counts as that where an infinity times 0 would give NaN.
__device__ __forceinline__ float activate(int act, float z, float cap)
{
    if (act == TT_ACT_RELU) return z < 0.f ? 0.f : z;
    if (act == TT_ACT_GELU) {
        float e;
        const float q = normal_tail(z, e);
        return (z < -1e30f ? -1e30f : z) * (z > 0.f ? 1.f - q : q);
    }
    if (act == TT_ACT_SILU) {
        const float e = expf(-fabsf(z));
        return (z < -1e30f ? -1e30f : z) * ((z < 0.f ? e : 1.f) * rcp(1.f + e));
    }
    if (act == TT_ACT_SOFTCAP) return cap * tanhf(z / cap);
    return z;
}

// act'(z), without differences of nearly equal numbers where it is small
__device__ __forceinline__ float slope(int act, float z, float cap)
{
    if (act == TT_ACT_RELU) return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
    if (act == TT_ACT_GELU) {
        float e;
        const float q = normal_tail(z, e), c = z > 100.f ? 100.f : z < -100.f ? -100.f : z;
        return fmaf(c * 0.39894228f, e, z > 0.f ? 1.f - q : q);
    }
    if (act == TT_ACT_SILU) {
        const float c = z > 1e30f ? 1e30f : z < -1e30f ? -1e30f : z;
        const float e = expf(-fabsf(c)), by = rcp(1.f + e);
        const float p = (c < 0.f ? e : 1.f) * by, q = (c < 0.f ? 1.f : e) * by;   // q = 1 - p
        return p * fmaf(c, q, 1.f);
    }
    if (act == TT_ACT_SOFTCAP) {       // 1 - tanh^2(u) = 4 e^-2u / (1 + e^-2u)^2
        const float e = expf(-2.f * fabsf(z / cap)), d = rcp(1.f + e);
        return 4.f * e * d * d;
    }
    return 1.f;
}

__device__ __forceinline__ float load_any(const void* p, int type, int64_t i)
{
    if (type == TT_BF16) return to_f32(((const __nv_bfloat16*)p)[i]);
    if (type == TT_F16) return to_f32(((const __half*)p)[i]);
    return ((const float*)p)[i];
}
__device__ __forceinline__ void store_any(void* p, int type, int64_t i, float x)
{
    if (type == TT_BF16) ((__nv_bfloat16*)p)[i] = from_f32<__nv_bfloat16>(x);
    else if (type == TT_F16) ((__half*)p)[i] = from_f32<__half>(x);
    else ((float*)p)[i] = x;
}

// What becomes of a sum s for row r and column c of the result:
//   z = s + bias[c];  pre[r][c] = z;  out[r][c] = act(z) + residual[r][c]
// each rounded once to its type.  The gradient of the table leaves `skip_row` out: its s counts as 0.
struct Epilogue {
    void* out;
    const void* residual;     // may be out itself: each value is read and then written by one thread
    void* pre;
    const void* bias;
    int64_t out_stride, residual_stride, pre_stride;
    int64_t skip_row;
    int32_t out_type, residual_type, pre_type, bias_type;
    int32_t act;
    float cap;
};
__device__ __forceinline__ void finish(const Epilogue& e, int64_t r, int64_t c, float s)
{
    float z = r == e.skip_row ? 0.f : s;
    if (e.bias) z += load_any(e.bias, e.bias_type, c);
    if (e.pre) store_any(e.pre, e.pre_type, r * e.pre_stride + c, z);
    float y = activate(e.act, z, e.cap);
    if (e.residual) y += load_any(e.residual, e.residual_type, r * e.residual_stride + c);
    store_any(e.out, e.out_type, r * e.out_stride + c, y);
}

// A matrix in memory: value (i, k) lies at p[i * si + k * sk].
struct Matrix {
    const void* p;
    int64_t si, sk;
    int32_t type;
};
// An upstream gradient: values of `up` times the slope at the values of `pre` (both row-major; pre may be null).
struct Upstream {
    const void* up;
    const void* pre;
    int64_t up_stride, pre_stride;
    int32_t up_type, pre_type;
    int32_t act;
    float cap;
};
__device__ __forceinline__ float upstream(const Upstream& u, int64_t r, int64_t c)
{
    float d = load_any(u.up, u.up_type, r * u.up_stride + c);
    if (u.act != TT_ACT_NONE) d *= slope(u.act, load_any(u.pre, u.pre_type, r * u.pre_stride + c), u.cap);
    return d;
}

}  // namespace tt
