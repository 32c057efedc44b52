// cbq_launch.cuh -- launches of the operators between and behind the products.
#pragma once

#include <cuda_runtime.h>

namespace cbq {

// Launches kernel<<<grid, threads, smem>>> as a programmatic dependent of the
// work ahead, in clusters of `cluster` blocks along the grid's y.
template <typename... P, typename... A>
inline cudaError_t launch_clusters(void (*kernel)(P...), dim3 grid, int cluster, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = at[1].val.clusterDim.z = 1;
    at[1].val.clusterDim.y = (unsigned)cluster;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kernel, (P)args...) : e;
}
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    return launch_clusters(kernel, grid, 1, threads, smem, s, args...);
}

}  // namespace cbq
