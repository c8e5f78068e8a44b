// Launch helpers of the context-free calls: programmatic dependent launches and per-device set-up.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace kvo {

// Programmatic dependent launch: the kernel starts while the one before it on the stream ends, and calls
// grid_wait (which returns once that kernel has completed) before it reads or writes anything.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Host: launch as a programmatic dependent, in clusters of `cluster` CTAs (0: none).
template <typename... P, typename... Q>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s,
                                    int cluster, const Q&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Host: true once per device for each `done` mask (function attributes are set per device).
inline bool first_on_device(std::atomic<uint64_t>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev > 63) return true;
    return !(done.load(std::memory_order_relaxed) >> dev & 1);
}
inline void mark_on_device(std::atomic<uint64_t>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev <= 63) done.fetch_or(1ull << dev, std::memory_order_relaxed);
}

}  // namespace kvo
