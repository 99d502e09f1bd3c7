// Launch of the small kernels of the language-model operators.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

namespace sg {

// A launch that may begin while the kernel before it in the stream ends
// (griddepcontrol.wait orders its memory accesses).
template <class... P, class... A>
cudaError_t launch(void (*fn)(P...), int64_t blocks, dim3 threads, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(std::max<int64_t>(1, blocks)));
    cfg.blockDim = threads;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, P(args)...);
}

}  // namespace sg
