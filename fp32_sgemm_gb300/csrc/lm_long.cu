// Gradients of 16-bit operands whose contraction (a group's rows, the tokens, a
// piece of the vocabulary) may be long, summed in runs (see lm_mma.cuh).
#include "lm_mma.cuh"

namespace sg {
LmKernel lm_weight_grad_kernel_long(int size) {
    if (size == 1) return lm_kernel_info<LmMid, true, true, kRagK, kEpiRows, kLong>();
    return lm_kernel_info<LmBig, true, true, kRagK, kEpiRows, kLong>();
}
LmKernel lm_rows_kernel_long(bool big, bool a_mn) {
    if (a_mn) return lm_kernel_info<LmBig, true, true, kRagNone, kEpiRows, kLong>();
    if (big) return lm_kernel_info<LmBig, false, true, kRagNone, kEpiRows, kLong>();
    return lm_kernel_info<LmWide, false, true, kRagNone, kEpiRows, kLong>();
}
}  // namespace sg
