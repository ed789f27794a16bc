// The table as a matrix: activations, what is done to a sum of products, and the kernels' arguments.
#pragma once

#include "roots.cuh"

namespace tt {

inline bool activation_known(int a) { return a >= TT_ACT_NONE && a <= TT_ACT_SOFTCAP; }

// 2^(hi + lo) for hi <= 0 and a small lo: what the rounding of hi has lost, so that far tails are right in relative terms
__device__ __forceinline__ F2 exp2_sum(F2 hi, F2 lo)
{
    F2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(hi.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(hi.y));
    return fma2(mul2(e, lo), both(0.69314718f), e);
}
constexpr float kLog2e = 1.4426950216293335f, kLog2eRest = 1.9259629911266175e-8f;     // their sum is log2(e)
__device__ __forceinline__ float magnitude_to(float z, float most)     // NaN stays NaN
{
    float w;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(w) : "f"(fabsf(z)), "f"(most));
    return w;
}
// e^-w for w >= 0
__device__ __forceinline__ F2 exp_minus(F2 w)
{
    const F2 hi = mul2(w, both(-kLog2e));
    return exp2_sum(hi, fma2(w, both(-kLog2eRest), fma2(w, both(-kLog2e), {-hi.x, -hi.y})));
}

// Phi(-w), the normal distribution function's tail, and e = exp(-w^2 / 2), for 0 <= w <= 40.  With x = w / sqrt(2),
// Phi(-w) = e erfcx(x) / 2, and erfcx(x) = exp(x^2) erfc(x) falls smoothly from 1 like 1 / x: a polynomial of t = 1 / (1 + 0.4 x)
// without a constant term, fitted to the least relative error, is within 1.4e-7 of it for all x >= 0.
__device__ __forceinline__ F2 normal_tail(F2 w, F2& e)
{
    const F2 s = mul2(w, w), s_lost = fma2(w, w, {-s.x, -s.y}), hi = mul2(s, both(-0.5f * kLog2e));
    F2 lo = fma2(s, both(-0.5f * kLog2e), {-hi.x, -hi.y});
    lo = fma2(s, both(-0.5f * kLog2eRest), lo);
    e = exp2_sum(hi, fma2(s_lost, both(-0.5f * kLog2e), lo));
    const F2 d = fma2(w, both(0.4f * 0.70710678f), both(1.f)), t = {rcp(d.x), rcp(d.y)};
    // (constants of single instructions need no register, those of paired ones two)
    auto poly = [](float t) {
        float p = 0.050265081f;
        p = fmaf(p, t, -0.18291025f);
        p = fmaf(p, t, 0.16909297f);
        p = fmaf(p, t, -0.0056056734f);
        p = fmaf(p, t, 0.14142445f);
        p = fmaf(p, t, 0.16854656f);
        p = fmaf(p, t, 0.20784137f);
        p = fmaf(p, t, 0.22566977f);
        return fmaf(p, t, 0.22567585f);
    };
    const F2 p = {poly(t.x), poly(t.y)};
    return mul2(mul2(mul2(e, both(0.5f)), t), p);
}

__device__ __forceinline__ float not_below_zero(float z)     // NaN stays NaN
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(0.f));
    return r;
}
// act(z) for a result of 16 bits, within 2^-15 of it: gelu's polynomial is within 5.2e-6, and the two roundings of an exponent
// below 2^7 leave 1.0e-5.
__device__ __forceinline__ float activate_coarse(int act, float z, float cap)
{
    if (act == TT_ACT_GELU) {
        const float w = fminf(fabsf(z), 13.f), t = rcp(fmaf(0.44f * 0.70710678f, w, 1.f));
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(w * (-0.5f * kLog2e) * w));
        float p = -0.14610514f;
        p = fmaf(p, t, 0.35065132f);
        p = fmaf(p, t, 0.0407319f);
        p = fmaf(p, t, 0.26358627f);
        p = fmaf(p, t, 0.24256945f);
        p = fmaf(p, t, 0.24856104f);
        return fmaf(-w, 0.5f * e * t * p, not_below_zero(z));
    }
    if (act == TT_ACT_SILU) {
        const float w = fminf(fabsf(z), 100.f);
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(w * -kLog2e));
        return fmaf(-w * e, rcp(1.f + e), not_below_zero(z));
    }
    if (act == TT_ACT_SOFTCAP) return cap * tanhf(z / cap);
    return act == TT_ACT_RELU ? not_below_zero(z) : z;
}

// act(z) of two values; infinities take their limits, and NaN stays NaN
__device__ __forceinline__ F2 activate(int act, F2 z, float cap)
{
    if (act == TT_ACT_RELU) return {not_below_zero(z.x), not_below_zero(z.y)};
    if (act == TT_ACT_GELU) {       // z Phi(z) = max(z, 0) - |z| Phi(-|z|)
        const F2 w = {magnitude_to(z.x, 40.f), magnitude_to(z.y, 40.f)};
        F2 e;
        const F2 q = normal_tail(w, e);
        return fma2({-w.x, -w.y}, q, {not_below_zero(z.x), not_below_zero(z.y)});
    }
    if (act == TT_ACT_SILU) {       // z / (1 + e^-z) = max(z, 0) - |z| e^-|z| / (1 + e^-|z|)
        const F2 w = {magnitude_to(z.x, 100.f), magnitude_to(z.y, 100.f)}, e = exp_minus(w), d = add2(e, both(1.f));
        return fma2(mul2({-w.x, -w.y}, e), {rcp(d.x), rcp(d.y)}, {not_below_zero(z.x), not_below_zero(z.y)});
    }
    if (act == TT_ACT_SOFTCAP) return {cap * tanhf(z.x / cap), cap * tanhf(z.y / cap)};
    return z;
}

// act'(z) of two values, without differences of nearly equal numbers where it is small
__device__ __forceinline__ F2 slope(int act, F2 z, float cap)
{
    if (act == TT_ACT_RELU) return {z.x > 0.f ? 1.f : z.x <= 0.f ? 0.f : z.x, z.y > 0.f ? 1.f : z.y <= 0.f ? 0.f : z.y};
    if (act == TT_ACT_GELU) {       // Phi(z) + z phi(z); of -z it is 1 less that of z
        const F2 w = {magnitude_to(z.x, 40.f), magnitude_to(z.y, 40.f)};
        F2 e;
        const F2 q = normal_tail(w, e), d = fma2(mul2(w, both(-0.39894228f)), e, q);
        return {z.x > 0.f ? 1.f - d.x : d.x, z.y > 0.f ? 1.f - d.y : d.y};
    }
    if (act == TT_ACT_SILU) {       // p (1 + z (1 - p)) with p = 1 / (1 + e^-z); likewise
        const F2 w = {magnitude_to(z.x, 100.f), magnitude_to(z.y, 100.f)}, e = exp_minus(w), d = add2(e, both(1.f));
        const F2 p = {rcp(d.x), rcp(d.y)}, q = mul2(e, p);
        const F2 v = mul2(q, fma2({-w.x, -w.y}, p, both(1.f)));
        return {z.x > 0.f ? 1.f - v.x : v.x, z.y > 0.f ? 1.f - v.y : v.y};
    }
    if (act == TT_ACT_SOFTCAP) {    // 1 - tanh^2(u) = 4 e^-2u / (1 + e^-2u)^2
        const F2 e = exp_minus({magnitude_to(2.f * (z.x / cap), 200.f), magnitude_to(2.f * (z.y / cap), 200.f)}), d = add2(e, both(1.f));
        const F2 p = {rcp(d.x), rcp(d.y)};
        return mul2(mul2(mul2(e, both(4.f)), p), p);
    }
    return both(1.f);
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

}  // namespace tt
