// What the host side of the 4-bit products and their kernel share.
#pragma once

#include <cstddef>
#include <cstdint>

namespace sg {

struct W4Args {
    int N, K, tokens;          // rows of W, columns, rows of x in this launch
    int k_slice;               // columns per blockIdx.y (a multiple of 256)
    const void *X;
    int64_t ldx;
    int x_vec;                 // rows of x take 16-byte loads
    int x_pitch;               // bytes of a staged row of x
    const uint8_t *Q;
    int64_t ldq;
    const void *scales;
    int64_t lds;
    const uint8_t *zeros;
    int64_t ldz;
    int s_vec, z_vec;          // a step's scales / zero points of a row in one vector load
    void *Y;
    int64_t ldy;
    float *part;               // [slice][token][ld_part] FP32, or NULL for Y itself
    int64_t ld_part;
    uint32_t *err;
    uint64_t timeout_ns;
    int withhold;
};

// nb: blocks of 8 columns (1, 2 or 4); alone: one CTA has an SM for itself.
const void *w4_kernel_f32(int group, int nb, bool zeros, bool alone);
const void *w4_kernel_f16(int group, int nb, bool zeros, bool alone);
const void *w4_kernel_bf16(int group, int nb, bool zeros, bool alone);
constexpr int kW4Stages = 4;                              // of 2 KB, per warp
constexpr int w4_warps(int nb, bool alone) { return alone && nb < 4 ? 16 : 8; }
// Shared memory beside the staged x: rings, the warps' sums twice, barriers.
inline size_t w4_fixed_smem(int nb, bool alone) {
    return 1024 + size_t(w4_warps(nb, alone)) * (kW4Stages * (2048 + 8) + 2 * nb * 512);
}

}  // namespace sg
