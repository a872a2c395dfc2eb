// fa_launch.h — launching a kernel that waits for the grid before it by itself.
#pragma once

#include <cuda_runtime.h>

namespace fa {

// Launch with programmatic stream serialization: the kernel waits for the grid
// before it in the stream (griddep_wait) before it touches global memory.
// `cluster`: CTAs of a cluster (1: none), a divisor of the grid.
template <typename... P, typename... A>
cudaError_t launch_dependent_clusters(void (*kernel)(P...), dim3 grid, unsigned cluster, unsigned threads, size_t smem,
                                      cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                             A... args) {
    return launch_dependent_clusters(kernel, grid, 1u, threads, smem, stream, args...);
}

}  // namespace fa
