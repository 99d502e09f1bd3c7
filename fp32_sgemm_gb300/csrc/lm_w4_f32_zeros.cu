// 4-bit products, x of type f32, zero points (see lm_w4.cuh).
#include "lm_w4.cuh"

namespace sg {
const void *w4_kernel_f32_zeros(int group, int nb, bool alone) {
    return w4_kernel_by_group<0, true>(group, nb, alone);
}
}  // namespace sg
