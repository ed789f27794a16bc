// The table as a matrix: activations, what is done to a sum of products, and the kernels' arguments.
#pragma once

#include "types.cuh"

namespace tt {

inline bool activation_known(int a) { return a >= TT_ACT_NONE && a <= TT_ACT_SOFTCAP; }

// act(z).  Values beyond 1e30 in magnitude count as that where an infinity times 0 would give NaN.
__device__ __forceinline__ float activate(int act, float z, float cap)
{
    if (act == TT_ACT_RELU) return z < 0.f ? 0.f : z;
    if (act == TT_ACT_GELU) return (z < -1e30f ? -1e30f : z) * normcdff(z);
    if (act == TT_ACT_SILU) {
        const float e = expf(-fabsf(z));
        return (z < -1e30f ? -1e30f : z) * ((z < 0.f ? e : 1.f) / (1.f + e));
    }
    if (act == TT_ACT_SOFTCAP) return cap * tanhf(z / cap);
    return z;
}

// act'(z), without differences of nearly equal numbers where it is small
__device__ __forceinline__ float slope(int act, float z, float cap)
{
    if (act == TT_ACT_RELU) return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
    if (act == TT_ACT_GELU) {
        const float c = z > 100.f ? 100.f : z < -100.f ? -100.f : z;
        return normcdff(c) + c * expf(-0.5f * c * c) * 0.3989422804014327f;
    }
    if (act == TT_ACT_SILU) {
        const float c = z > 1e30f ? 1e30f : z < -1e30f ? -1e30f : z;
        const float e = expf(-fabsf(c)), by = 1.f / (1.f + e);
        const float p = (c < 0.f ? e : 1.f) * by, q = (c < 0.f ? 1.f : e) * by;   // q = 1 - p
        return p * (1.f + c * q);
    }
    if (act == TT_ACT_SOFTCAP) {       // 1 - tanh^2(u) = 4 e^-2u / (1 + e^-2u)^2
        const float e = expf(-2.f * fabsf(z / cap)), d = 1.f + e;
        return 4.f * e / (d * d);
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
