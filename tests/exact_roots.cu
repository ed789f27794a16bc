// Counts the values at which minus_root2 and inverse differ from the correctly rounded square root and
// reciprocal: all 2^23 mantissas of the exponents first .. last.
#include "roots.cuh"

using namespace tt;

namespace {

struct Found {
    unsigned long long count;
    float example;
};

template <bool kRoot>
__global__ void __launch_bounds__(256) compare(int first, Found* found)
{
    const uint32_t mantissa = blockIdx.x * 256u + threadIdx.x, exponent = (uint32_t)(127 + first + (int)blockIdx.y);
    const float x = __uint_as_float(exponent << 23 | mantissa);
    bool same;
    if constexpr (kRoot) {
        // the other value of the pair is another one, as it is in use
        const float y = __uint_as_float(exponent << 23 | (mantissa ^ 0x2aaaaau));
        const F2 got = minus_root2({-x, -y});
        same = got.x == -__fsqrt_rn(x) && got.y == -__fsqrt_rn(y);
    } else {
        same = inverse(x) == __frcp_rn(x);
    }
    if (!same && atomicAdd(&found->count, 1ull) == 0) found->example = x;
}

template <bool kRoot>
long long run(int first, int last, float* example)
{
    if (first < -126 || last > 127 || last < first) return -1;
    Found* at = nullptr;
    Found got = {0, 0.f};
    if (cudaMalloc((void**)&at, sizeof(Found)) != cudaSuccess) return -1;
    bool ok = cudaMemcpy(at, &got, sizeof(got), cudaMemcpyHostToDevice) == cudaSuccess;
    compare<kRoot><<<dim3((1u << 23) / 256u, (unsigned)(last - first + 1)), 256>>>(first, at);
    ok = ok && cudaGetLastError() == cudaSuccess && cudaMemcpy(&got, at, sizeof(got), cudaMemcpyDeviceToHost) == cudaSuccess;
    cudaFree(at);
    if (!ok) return -1;
    *example = got.example;
    return (long long)got.count;
}

}  // namespace

extern "C" long long different_roots(int first, int last, float* example) { return run<true>(first, last, example); }
extern "C" long long different_reciprocals(int first, int last, float* example) { return run<false>(first, last, example); }
