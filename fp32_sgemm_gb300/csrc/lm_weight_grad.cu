// Gradients of the groups' matrices (see lm_mma.cuh): the contraction runs
// over the rows of a group, both operands are read with that index outermost.
#include "lm_mma.cuh"

namespace sg {
LmKernel lm_weight_grad_kernel_long(int size);

LmKernel lm_weight_grad_kernel(int size, bool f32, bool lengthy) {
    if (f32) {
        if (size == 1) return lm_kernel_info<LmMid, true, true, kRagK, kEpiRows, kPlanes>();
        return lm_kernel_info<LmBig, true, true, kRagK, kEpiRows, kPlanes>();
    }
    if (lengthy) return lm_weight_grad_kernel_long(size);
    if (size == 1) return lm_kernel_info<LmMid, true, true, kRagK, kEpiRows, kPlain>();
    return lm_kernel_info<LmBig, true, true, kRagK, kEpiRows, kPlain>();
}
}  // namespace sg
