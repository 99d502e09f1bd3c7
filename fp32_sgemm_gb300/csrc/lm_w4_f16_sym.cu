// 4-bit products, x of type f16, no zero points (see lm_w4.cuh).
#include "lm_w4.cuh"

namespace sg {
const void *w4_kernel_f16_zeros(int group, int nb, bool alone);

const void *w4_kernel_f16(int group, int nb, bool zeros, bool alone) {
    return zeros ? w4_kernel_f16_zeros(group, nb, alone) : w4_kernel_by_group<1, false>(group, nb, alone);
}
}  // namespace sg
