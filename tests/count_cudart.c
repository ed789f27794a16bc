/* A CUDA runtime for tests without a device, which counts what a handle's making asks of it: host memory stands in for the device's,
 * and every launch is refused. */
#include <cuda_runtime_api.h>
#include <stdlib.h>
#include <string.h>

static int allocations, waits, questions;

/* allocations, waits for a stream and questions about a kernel since the last call */
void count_take(int* out)
{
    out[0] = allocations;
    out[1] = waits;
    out[2] = questions;
    allocations = waits = questions = 0;
}

cudaError_t cudaGetDevice(int* device) { *device = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* value, enum cudaDeviceAttr attr, int device)
{
    (void)attr; (void)device;
    *value = 148;
    return cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t bytes) { ++allocations; *p = malloc(bytes); return *p ? cudaSuccess : cudaErrorMemoryAllocation; }
cudaError_t cudaFree(void* p) { free(p); return cudaSuccess; }
cudaError_t cudaMemset(void* p, int value, size_t bytes) { memset(p, value, bytes); return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t s) { (void)s; ++waits; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute attr, int value) { (void)f; (void)attr; (void)value; return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* clusters, const void* f, const cudaLaunchConfig_t* c)
{
    (void)f; (void)c;
    ++questions;
    *clusters = 1;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernel(const void* f, dim3 g, dim3 b, void** a, size_t m, cudaStream_t s)
{
    (void)f; (void)g; (void)b; (void)a; (void)m; (void)s;
    return cudaErrorNotSupported;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** a) { (void)c; (void)f; (void)a; return cudaErrorNotSupported; }
cudaError_t cudaGetLastError(void) { return cudaErrorNotSupported; }
