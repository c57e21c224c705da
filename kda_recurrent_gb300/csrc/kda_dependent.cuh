// Launches that overlap the end of the launch before them on the stream (programmatic dependent launch).
//
// A kernel launched so may start while earlier work on its stream still runs. Every thread therefore passes
// wait_for_prior before it touches global memory, the call's inputs included: only that wait makes visible
// what was written before, by the launch before directly and, since that one waited too, by all earlier
// ones. allow_next lets the next launch start at any time, which then waits in the same way. A launch's
// latency and its kernel's set-up so lie behind the kernel before it.
#pragma once

#include <cuda_runtime.h>

namespace kda {

__device__ __forceinline__ void wait_for_prior() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_clusters(unsigned cluster, void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                            const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream, const A &...args) {
    return launch_clusters(1, kernel, grid, block, smem, stream, args...);
}

}  // namespace kda
