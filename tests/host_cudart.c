/* A CUDA runtime for tests without a device: handles can be made, host memory stands in for the device's, and every
 * launch is refused.  For the checks that the library makes on the host before any device work. */
#include <cuda_runtime_api.h>
#include <stdlib.h>
#include <string.h>

cudaError_t cudaGetDevice(int* device) { *device = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* value, enum cudaDeviceAttr attr, int device)
{
    (void)attr; (void)device;
    *value = 148;
    return cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t bytes) { *p = malloc(bytes); return *p ? cudaSuccess : cudaErrorMemoryAllocation; }
cudaError_t cudaFree(void* p) { free(p); return cudaSuccess; }
cudaError_t cudaMemset(void* p, int value, size_t bytes) { memset(p, value, bytes); return cudaSuccess; }
cudaError_t cudaMemsetAsync(void* p, int value, size_t bytes, cudaStream_t s) { (void)p; (void)value; (void)bytes; (void)s; return cudaErrorNotSupported; }
cudaError_t cudaStreamSynchronize(cudaStream_t s) { (void)s; return cudaSuccess; }
cudaError_t cudaLaunchKernel(const void* f, dim3 g, dim3 b, void** a, size_t m, cudaStream_t s)
{
    (void)f; (void)g; (void)b; (void)a; (void)m; (void)s;
    return cudaErrorNotSupported;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** a) { (void)c; (void)f; (void)a; return cudaErrorNotSupported; }
cudaError_t cudaGetLastError(void) { return cudaErrorNotSupported; }
