// Launches that overlap the end of the kernel before them on the stream: the
// blocks may be placed while that kernel finishes, and every thread calls
// after_previous() before it touches memory, which returns once that kernel is
// done and its writes are visible.  Worth 0.5 to 1 us a launch between the
// short kernels of a decode step.
#pragma once

#include <cuda_runtime.h>

namespace csa_dev {

__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// `cluster` blocks to a cluster.
template <typename... P, typename... A>
inline cudaError_t launch_clusters_after_previous(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                                                  cudaStream_t stream, int cluster, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = (unsigned)cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    (void)cudaLaunchKernelEx(&cfg, kernel, args...);
    return cudaGetLastError();  // and taken, or the next launch would report it too
}

template <typename... P, typename... A>
inline cudaError_t launch_after_previous(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                                         cudaStream_t stream, A... args) {
    return launch_clusters_after_previous(kernel, grid, threads, smem, stream, 1, args...);
}

}  // namespace csa_dev
