// Grouped products of 16-bit operands with a long contraction, summed in runs
// (see lm_mma.cuh).
#include "lm_mma.cuh"

namespace sg {
LmKernel lm_grouped_kernel_long(int size, bool w_mn) {
    if (w_mn) {
        if (size == 0) return lm_kernel_info<LmThin, true, false, kRagN, kEpiCols, kLong>();
        if (size == 1) return lm_kernel_info<LmMid, true, false, kRagN, kEpiCols, kLong>();
        return lm_kernel_info<LmBig, true, false, kRagN, kEpiCols, kLong>();
    }
    if (size == 0) return lm_kernel_info<LmThin, false, false, kRagN, kEpiCols, kLong>();
    if (size == 1) return lm_kernel_info<LmMid, false, false, kRagN, kEpiCols, kLong>();
    return lm_kernel_info<LmBig, false, false, kRagN, kEpiCols, kLong>();
}
}  // namespace sg
