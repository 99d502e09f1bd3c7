// Products of the vocabulary cross entropy for 16-bit operands (see
// lm_mma.cuh): the logits of a tile live in tensor memory only.
#include "lm_mma.cuh"

namespace sg {
LmKernel lm_lse_kernel32(bool big);
LmKernel lm_dlogits_kernel32(bool big);
LmKernel lm_rows_kernel32(bool big, bool a_mn);
LmKernel lm_rows_kernel_long(bool big, bool a_mn);

LmKernel lm_lse_kernel(bool big, bool f32) {
    if (f32) return lm_lse_kernel32(big);
    if (big) return lm_kernel_info<LmBigBare, false, false, kRagNone, kEpiLse, kRuns>();
    return lm_kernel_info<LmWide, false, false, kRagNone, kEpiLse, kRuns>();
}
LmKernel lm_dlogits_kernel(bool big, bool f32) {
    if (f32) return lm_dlogits_kernel32(big);
    if (big) return lm_kernel_info<LmBigBare, false, false, kRagNone, kEpiDLogits, kRuns>();
    return lm_kernel_info<LmWide, false, false, kRagNone, kEpiDLogits, kRuns>();
}
LmKernel lm_rows_kernel(bool big, bool a_mn, bool f32, bool lengthy) {
    if (f32) return lm_rows_kernel32(big, a_mn);
    if (lengthy) return lm_rows_kernel_long(big, a_mn);
    if (a_mn) return lm_kernel_info<LmBig, true, true, kRagNone, kEpiRows, kPlain>();
    if (big) return lm_kernel_info<LmBig, false, true, kRagNone, kEpiRows, kPlain>();
    return lm_kernel_info<LmWide, false, true, kRagNone, kEpiRows, kPlain>();
}
}  // namespace sg
