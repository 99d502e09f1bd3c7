// Grouped products of FP32 operands, held as three bf16 planes each (see
// lm_mma.cuh): six plane products per block, summed block by block in FP32.
#include "lm_mma.cuh"

namespace sg {
LmKernel lm_grouped_kernel16(int size, bool w_mn);
LmKernel lm_grouped_kernel_long(int size, bool w_mn);

LmKernel lm_grouped_kernel(int size, bool w_mn, bool f32, bool lengthy) {
    if (!f32) return lengthy ? lm_grouped_kernel_long(size, w_mn) : lm_grouped_kernel16(size, w_mn);
    if (w_mn) {
        if (size == 0) return lm_kernel_info<LmThin, true, false, kRagN, kEpiCols, kPlanes>();
        if (size == 1) return lm_kernel_info<LmMid, true, false, kRagN, kEpiCols, kPlanes>();
        return lm_kernel_info<LmBig, true, false, kRagN, kEpiCols, kPlanes>();
    }
    if (size == 0) return lm_kernel_info<LmThin, false, false, kRagN, kEpiCols, kPlanes>();
    if (size == 1) return lm_kernel_info<LmMid, false, false, kRagN, kEpiCols, kPlanes>();
    return lm_kernel_info<LmBig, false, false, kRagN, kEpiCols, kPlanes>();
}
}  // namespace sg
