// launch.h -- launches of the operators' kernels as programmatic dependents:
// the launch itself, and what a kernel does before its griddepcontrol.wait,
// overlap the end of the kernel before it on the stream. Every thread of such a
// kernel waits before it reads or writes global memory, so that the kernel is
// not done before its predecessor is.
#pragma once

#include <cuda_runtime.h>

namespace kvevict {

template <typename P>
cudaError_t launch_dependent(void (*kernel)(P), unsigned grid, unsigned block, size_t smem, cudaStream_t st, const P &params)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(grid, 1, 1);
    lc.blockDim = dim3(block, 1, 1);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = &attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, params);
}

}  // namespace kvevict
