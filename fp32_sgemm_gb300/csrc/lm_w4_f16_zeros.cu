// 4-bit products, x of type f16, zero points (see lm_w4.cuh).
#include "lm_w4.cuh"

namespace sg {
const void *w4_kernel_f16_zeros(int group, int nb, bool alone) {
    return w4_kernel_by_group<1, true>(group, nb, alone);
}
}  // namespace sg
