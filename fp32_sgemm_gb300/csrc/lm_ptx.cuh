// PTX wrappers the language-model kernels share beside those of ptx.cuh.
#pragma once

#include "ptx.cuh"

namespace sg {

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
    return is != 0;
}

}  // namespace sg
