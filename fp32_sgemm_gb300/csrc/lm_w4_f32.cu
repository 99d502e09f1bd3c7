// 4-bit products, x of type f32 (see lm_w4.cuh).
#include "lm_w4.cuh"

namespace sg {
const void *w4_kernel_f32(int group, int nb) { return w4_kernel_of<0>(group, nb); }
size_t w4_fixed_smem(int nb) { return kW4RingBytes + 2 * kW4Warps * nb * 512; }
}  // namespace sg
