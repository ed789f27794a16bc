/* Stands in front of the CUDA runtime in a test's process: another current device, or a device on which no cluster
 * fits, as the library is told of them.  Everything else is passed on. */
#define _GNU_SOURCE
#include <cuda_runtime_api.h>
#include <dlfcn.h>

static int other_device = -1, no_clusters = 0, cluster_launches = 0;

void fake_device(int device) { other_device = device; }
void fake_no_clusters(int on) { no_clusters = on; }
int fake_cluster_launches(void) { return cluster_launches; }

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

cudaError_t cudaOccupancyMaxActiveClusters(int* clusters, const void* kernel, const cudaLaunchConfig_t* config)
{
    cudaError_t (*f)(int*, const void*, const cudaLaunchConfig_t*) =
        (cudaError_t(*)(int*, const void*, const cudaLaunchConfig_t*))real("cudaOccupancyMaxActiveClusters");
    const cudaError_t e = f ? f(clusters, kernel, config) : cudaErrorNotSupported;
    if (e == cudaSuccess && no_clusters) *clusters = 0;
    return e;
}

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* config, const void* kernel, void** args)
{
    for (unsigned i = 0; i < config->numAttrs; ++i)
        if (config->attrs[i].id == cudaLaunchAttributeClusterDimension) {
            if (no_clusters) return cudaErrorInvalidClusterSize;
            ++cluster_launches;
        }
    cudaError_t (*f)(const cudaLaunchConfig_t*, const void*, void**) =
        (cudaError_t(*)(const cudaLaunchConfig_t*, const void*, void**))real("cudaLaunchKernelExC");
    return f ? f(config, kernel, args) : cudaErrorNotSupported;
}
