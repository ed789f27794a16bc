/* Stands in front of the CUDA runtime in a test's process: another current device, as the library is told of it.
 * Everything else is passed on. */
#define _GNU_SOURCE
#include <cuda_runtime_api.h>
#include <dlfcn.h>

static int other_device = -1;

void fake_device(int device) { other_device = device; }

static void* real(const char* name)
{
    void* lib = dlopen("libcudart.so.12", RTLD_NOW | RTLD_NOLOAD);
    return lib ? dlsym(lib, name) : 0;
}

cudaError_t cudaGetDevice(int* device)
{
    cudaError_t (*f)(int*) = (cudaError_t(*)(int*))real("cudaGetDevice");
    const cudaError_t e = f ? f(device) : cudaErrorNotSupported;
    if (e == cudaSuccess && other_device >= 0) *device = other_device;
    return e;
}
