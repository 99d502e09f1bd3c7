// 4-bit products, x of type f16 (see lm_w4.cuh).
#include "lm_w4.cuh"

namespace sg {
const void *w4_kernel_f16(int group, int nb, bool alone) { return w4_kernel_of<1>(group, nb, alone); }

}  // namespace sg
