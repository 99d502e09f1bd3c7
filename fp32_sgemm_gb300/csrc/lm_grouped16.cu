// Grouped products of 16-bit operands (see lm_mma.cuh): rows of the token
// matrix on the MMA's N side, the group's matrix on its M side.
#include "lm_mma.cuh"

namespace sg {
LmKernel lm_grouped_kernel16(int size, bool w_mn) {
    if (w_mn) {
        if (size == 0) return lm_kernel_info<LmThin, true, false, kRagN, kEpiCols, kPlain>();
        if (size == 1) return lm_kernel_info<LmMid, true, false, kRagN, kEpiCols, kPlain>();
        return lm_kernel_info<LmBig, true, false, kRagN, kEpiCols, kPlain>();
    }
    if (size == 0) return lm_kernel_info<LmThin, false, false, kRagN, kEpiCols, kPlain>();
    if (size == 1) return lm_kernel_info<LmMid, false, false, kRagN, kEpiCols, kPlain>();
    return lm_kernel_info<LmBig, false, false, kRagN, kEpiCols, kPlain>();
}
}  // namespace sg
