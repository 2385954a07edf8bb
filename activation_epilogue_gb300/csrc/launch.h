// Launching a kernel as a programmatic dependent of the stream's previous work (internal).
// The kernel may start while that work still runs and calls grid_dependency_wait() in every
// thread before it touches memory.  cluster > 1: in clusters of that many blocks (grid is a
// multiple of it).
#pragma once

#include <atomic>
#include <cuda_runtime.h>

namespace gemm_epi {

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int grid, int threads, int smem,
                             cudaStream_t stream, int cluster, const Args&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

// Let a kernel use up to `bytes` of dynamic shared memory on the current device; `done` (one
// bit per device, static beside the kernel's launch) makes it a single call per device.
template <typename Kernel>
cudaError_t allow_smem(Kernel* kernel, int bytes, std::atomic<unsigned long long>& done)
{
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t s = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (s == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return s;
}

}  // namespace gemm_epi
