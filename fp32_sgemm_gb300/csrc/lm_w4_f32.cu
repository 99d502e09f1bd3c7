// 4-bit products, x of type f32 (see lm_w4.cuh).
#include "lm_w4.cuh"

namespace sg {
const void *w4_kernel_f32(int group, int nb, bool alone) { return w4_kernel_of<0>(group, nb, alone); }
}  // namespace sg
