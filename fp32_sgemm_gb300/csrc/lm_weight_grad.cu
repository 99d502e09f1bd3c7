// Gradients of the groups' matrices (see lm_mma.cuh): the contraction runs
// over the rows of a group, both operands are read with that index outermost.
#include "lm_mma.cuh"

namespace sg {
LmKernel lm_weight_grad_kernel(int size, bool f32) {
    if (f32) {
        if (size == 1) return lm_kernel_info<LmMid, true, true, kRagK, kEpiRows, true>();
        return lm_kernel_info<LmBig, true, true, kRagK, kEpiRows, true>();
    }
    if (size == 1) return lm_kernel_info<LmMid, true, true, kRagK, kEpiRows, false>();
    return lm_kernel_info<LmBig, true, true, kRagK, kEpiRows, false>();
}
}  // namespace sg
