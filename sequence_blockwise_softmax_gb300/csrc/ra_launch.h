// ra_launch.h -- launching a kernel that may start before its predecessor ends.
#pragma once
#include <cuda_runtime.h>

#include "ra_internal.h"

namespace ra {

// Launch `kern` so that its blocks may start while the stream's previous kernel
// still runs (see pdl_wait in ra_device.cuh).
template <class... P, class... A>
inline cudaError_t launch_dependent(void (*kern)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                                    const A &...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// The same in clusters of `cluster` blocks.
template <class... P, class... A>
inline cudaError_t launch_dependent_clusters(void (*kern)(P...), unsigned cluster, unsigned grid, unsigned block,
                                             size_t smem, cudaStream_t stream, const A &...args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// A call's status from that of its launches.
inline ra_status launched(cudaError_t e) {
    if (e == cudaSuccess) return RA_OK;
    cudaGetLastError();      // reported here, not to the next caller
    return set_error(RA_ERR_CUDA, cudaGetErrorString(e));
}

}  // namespace ra
