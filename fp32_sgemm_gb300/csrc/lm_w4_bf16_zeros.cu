// 4-bit products, x of type bf16, zero points (see lm_w4.cuh).
#include "lm_w4.cuh"

namespace sg {
const void *w4_kernel_bf16_zeros(int group, int nb, bool alone) {
    return w4_kernel_by_group<2, true>(group, nb, alone);
}
}  // namespace sg
