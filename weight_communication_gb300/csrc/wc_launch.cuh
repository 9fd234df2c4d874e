// wc_launch.cuh -- launches that overlap the end of their predecessor in the
// stream, for calls of several short kernels.
//
// A kernel launched with launch_after() may start before its predecessor in
// the stream has ended, and calls wait_for_predecessor() before it touches any
// memory that the predecessor writes; a predecessor that calls
// let_successor_start() allows that as soon as all its CTAs have started, any
// other one when it ends.
#pragma once

#include <cuda_runtime.h>

namespace wc {

__device__ __forceinline__ void let_successor_start() {
    asm volatile("griddepcontrol.launch_dependents;");
}
__device__ __forceinline__ void wait_for_predecessor() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// `cluster`: CTAs of a cluster, along x.
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                         cudaStream_t stream, unsigned cluster, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
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
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace wc
