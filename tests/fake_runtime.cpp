// Stands in for the CUDA runtime calls of the library's host code (linked with
// --wrap), so that argument checks, workspace sizes and launches can be tested
// without a GPU: nothing is launched, copied or written.  A device is a number
// that fake_use sets; a kernel's raised shared-memory limit belongs to the
// device that was in use, as it does in the runtime, and a launch beyond it
// fails.
#include <cstdint>
#include <cstring>
#include <map>
#include <utility>

#include <cuda.h>
#include <cuda_runtime.h>

namespace {

int g_device = 0, g_failing = 0;
cudaError_t g_last = cudaSuccess;
std::map<std::pair<int, const void*>, int> g_smem;
int64_t g_launches = 0, g_blocks = 0;
int g_attributes = 0, g_queries = 0;

cudaError_t set(cudaError_t e) {
    if (e != cudaSuccess) g_last = e;
    return e;
}

cudaError_t launched(const void* f, dim3 grid, dim3 block, size_t smem) {
    if (grid.x == 0 || grid.y == 0 || grid.y > 65535 || block.x == 0 || block.x > 1024)
        return set(cudaErrorInvalidConfiguration);
    const auto it = g_smem.find({g_device, f});
    if (smem > (it == g_smem.end() ? 48u * 1024 : (size_t)it->second))
        return set(cudaErrorInvalidValue);
    ++g_launches;
    g_blocks = (int64_t)grid.x * grid.y * grid.z;
    return cudaSuccess;
}

CUresult encode(CUtensorMap* map, CUtensorMapDataType, cuuint32_t, void* base, const cuuint64_t*,
                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    memset(map, 0, sizeof(*map));
    return (uintptr_t)base % 16 ? CUDA_ERROR_INVALID_VALUE : CUDA_SUCCESS;
}

}  // namespace

extern "C" {

// device: 0 has 152 multiprocessors, device d 152 - 10 d.  failing: occupancy
// and attribute queries fail.
void fake_use(int device, int failing) {
    g_device = device;
    g_failing = failing;
}
int64_t fake_launches() { return g_launches; }
int64_t fake_blocks() { return g_blocks; }       // of the last launch
int fake_attribute_calls() { return g_attributes; }
int fake_queries() { return g_queries; }         // of occupancy

cudaError_t __wrap_cudaGetDevice(int* d) {
    *d = g_device;
    return cudaSuccess;
}
cudaError_t __wrap_cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int device) {
    *v = 152 - 10 * device;
    return g_failing ? set(cudaErrorUnknown) : cudaSuccess;
}
cudaError_t __wrap_cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int,
                                                                         size_t, unsigned) {
    ++g_queries;
    *n = 2;
    return g_failing ? set(cudaErrorUnknown) : cudaSuccess;
}
cudaError_t __wrap_cudaOccupancyMaxActiveClusters(int* n, const void*,
                                                  const cudaLaunchConfig_t* config) {
    ++g_queries;
    *n = (152 - 10 * g_device) / (int)config->gridDim.x;
    return g_failing ? set(cudaErrorUnknown) : cudaSuccess;
}
cudaError_t __wrap_cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int value) {
    ++g_attributes;
    if (g_failing) return set(cudaErrorUnknown);
    g_smem[{g_device, f}] = value;
    return cudaSuccess;
}
cudaError_t __wrap___cudaGetKernel(cudaKernel_t* k, const void* f) {
    *k = (cudaKernel_t)f;
    return cudaSuccess;
}
cudaError_t __wrap___cudaLaunchKernel(cudaKernel_t k, dim3 grid, dim3 block, void**, size_t smem,
                                      cudaStream_t) {
    return launched((const void*)k, grid, block, smem);
}
cudaError_t __wrap_cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
    return launched(f, c->gridDim, c->blockDim, c->dynamicSmemBytes);
}
cudaError_t __wrap_cudaGetLastError() {
    const cudaError_t e = g_last;
    g_last = cudaSuccess;
    return e;
}
cudaError_t __wrap_cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t __wrap_cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) {
    return cudaSuccess;
}
cudaError_t __wrap_cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned,
                                                    unsigned long long,
                                                    cudaDriverEntryPointQueryResult* found) {
    *p = (void*)encode;
    if (found) *found = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}

}  // extern "C"
