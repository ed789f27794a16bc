// Element types of the dense-table and AdamW kernels: fp32, bf16 and fp16 values moved as
// vectors and computed on in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <string.h>

#include "tt_common.cuh"

namespace tt {

inline int type_bytes(int t) { return t == TT_F32 ? 4 : 2; }
inline bool type_known(int t) { return t == TT_F32 || t == TT_BF16 || t == TT_F16; }

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// the one rounding of a result to its type (to nearest, ties to even)
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// N values at p, which is aligned to min(16, N * sizeof(T)) bytes
template <typename T, int N> struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Pack { T v[N]; };

template <int N, typename T>
__device__ __forceinline__ void store_pack(T* p, const float (&x)[N])
{
    Pack<T, N> q;
#pragma unroll
    for (int i = 0; i < N; ++i) q.v[i] = from_f32<T>(x[i]);
    *reinterpret_cast<Pack<T, N>*>(p) = q;
}

// Pairs of fp32 values in one register pair: one instruction for both.  The compiler fuses packed
// products and sums, .rn or not; where each is to be rounded on its own, a sum of products is written
// fma2(a, one, b) with a factor that it cannot see.
struct F2 { float x, y; };
__device__ __forceinline__ uint64_t bits2(F2 a) { uint64_t r; asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y)); return r; }
__device__ __forceinline__ F2 pair(uint64_t r) { F2 a; asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r)); return a; }
__device__ __forceinline__ F2 both(float x) { return {x, x}; }
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair(r);
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair(r);
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return pair(r);
}
// Kernels of one call are launched with leave to start while the one before still runs: each waits here until that
// one has ended and its writes can be read, which hides the launch.
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// a launch that may start while the kernel before it still runs
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), unsigned grid, unsigned threads, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.gridDim = dim3(grid);
    c.blockDim = dim3(threads);
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

// f(T()) for the C++ type of a known tt_dtype
template <typename F>
auto by_type(int t, F&& f)
{
    if (t == TT_BF16) return f(__nv_bfloat16());
    if (t == TT_F16) return f(__half());
    return f(float());
}

}  // namespace tt
