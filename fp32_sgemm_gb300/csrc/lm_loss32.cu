// Products of the vocabulary cross entropy for FP32 operands, each held as
// three bf16 planes (see lm_mma.cuh).
#include "lm_mma.cuh"

namespace sg {
LmKernel lm_lse_kernel32(bool big) {
    if (big) return lm_kernel_info<LmBig, false, false, kRagNone, kEpiLse, kPlanes>();
    return lm_kernel_info<LmMid, false, false, kRagNone, kEpiLse, kPlanes>();
}
LmKernel lm_dlogits_kernel32(bool big) {
    if (big) return lm_kernel_info<LmBig, false, false, kRagNone, kEpiDLogits, kPlanes>();
    return lm_kernel_info<LmMid, false, false, kRagNone, kEpiDLogits, kPlanes>();
}
LmKernel lm_rows_kernel32(bool big, bool a_mn) {
    if (a_mn) return lm_kernel_info<LmBig, true, true, kRagNone, kEpiRows, kPlanes>();
    if (big) return lm_kernel_info<LmBig, false, true, kRagNone, kEpiRows, kPlanes>();
    return lm_kernel_info<LmMid, false, true, kRagNone, kEpiRows, kPlanes>();
}
}  // namespace sg
