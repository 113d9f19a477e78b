// pdl.cuh -- launches that overlap with the end of the kernel before them in their stream (programmatic
// dependent launch).  A kernel launched with launch_overlapped may become resident while its predecessor still
// runs; it touches no memory before wait_primary(), which returns once every earlier kernel of the stream has
// completed and its writes are visible.  So results are those of plain launches; what overlaps is the launch
// itself (1.5 to 2.5 us between kernels that run for a few).
#pragma once

#include <cuda_runtime.h>

namespace dspark {

// Lets the next kernel of the stream be launched now, if it was launched with launch_overlapped.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_overlapped_clusters(void (*kernel)(P...), dim3 grid, int cluster, dim3 block, size_t smem, cudaStream_t s,
                                       A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A&&... args) {
    return launch_overlapped_clusters(kernel, grid, 1, block, smem, s, args...);
}

}  // namespace dspark
