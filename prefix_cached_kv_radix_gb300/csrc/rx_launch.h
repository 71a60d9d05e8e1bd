// Kernel launches that overlap the end of the kernel before them.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace rx {

// Launches with programmatic serialization: the grid may be set up while the last blocks of the kernel
// before it in the stream run, once all of those have started.  Every thread of such a kernel calls
// pdl_wait before it touches global memory or leaves, so that the kernel has finished only when all
// before it have.
template <class... P, class... A>
cudaError_t launch_pdl(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream, A&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace rx
