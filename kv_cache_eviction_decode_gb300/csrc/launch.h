// launch.h -- launches of the operators' kernels as programmatic dependents:
// the launch itself, and what a kernel does before its griddepcontrol.wait,
// overlap the end of the kernel before it on the stream. Every thread of such a
// kernel waits before it reads or writes global memory, so that the kernel is
// not done before its predecessor is.
#pragma once

#include <cuda_runtime.h>

namespace kvevict {

// cluster: CTAs of a cluster, 1 for none.
template <typename P>
cudaError_t launch_dependent(void (*kernel)(P), unsigned grid, unsigned block, size_t smem, cudaStream_t st, const P &params, unsigned cluster = 1)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(grid, 1, 1);
    lc.blockDim = dim3(block, 1, 1);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, kernel, params);
}

}  // namespace kvevict
