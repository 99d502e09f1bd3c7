// Kernels of the products in 8-bit integers with scales for each token and
// channel (lm_int8_quant.cu, lm_int8_rows.cu, lm_int8_mma.cu).
#pragma once

#include "lm_kernels.h"

namespace sg {

// Terms whose sum one FP32 accumulator holds exactly: 1024 * 128 * 128 = 2^24.
constexpr int kInt8Run = 1024;
// Most terms whose sum 32 bits hold: 131071 * 128 * 128 < 2^31.
constexpr int64_t kInt8MaxK = 131071;

// Rows of X as 8-bit integers (out16: the same integers in f16) and their
// scales.  from: sgemmDataType_t, or 3 for rows that are integers already
// (copied, no scales).  `cols` columns are written, those from K on as 0; in f16
// cols and the pitch are multiples of 8.  chained: see the kernel.
cudaError_t int8_quantize_launch(int from, const void *x, int64_t ldx, int64_t T, int64_t K, void *out, int64_t ldo,
                                 int64_t cols, bool out16, float *scales, bool chained, cudaStream_t s);

struct Int8Args {
    LmArgs lm;                       // M = N of the product, T, G, ends, C, ldc, out, tiles
    const float *x_scales;           // [T]
    const float *scales;             // [G][N]
    int32_t *row_group;              // [T], where parts of the contraction are joined later, or NULL
    // lm_int8_rows.cu
    const void *x;                   // [T][ldx]; integers: ldx a multiple of 16, base 16-byte aligned
    int64_t ldx;
    int from, x_vec;                 // sgemmDataType_t of x; numbers: rows take 16-byte loads
    const int8_t *w;
    int64_t ldw, stride_w;
    int K, k_slice, w_vec, early;    // early: the kernel before wrote x and its scales and nothing else
    int x_pitch;                     // bytes of a token's x in shared memory
};

// Tokens of a tile: 1, 2, 4 or 8; warps 8 (ks 1, 4 or 8) or 16 (ks 4, 8 or
// 16), ks of which share the contraction of 16 rows.
LmKernel int8_rows_kernel(int tokens, int warps, int ks);
// Bytes of one token's x, and of a CTA with x of `rows` tokens.
int64_t int8_rows_pitch(int tokens, int64_t k_slice);
int64_t int8_rows_smem(int tokens, int rows, int warps, int64_t k_slice, int64_t G);

// bn: rows of x in a tile at most; gran: columns of K in a block.
LmKernel int8_mma_kernel(bool wide);

// out = x_scales * scales * (sum of `splits` int32 planes), rounded to `out_type`;
// rows of no group (row_group < 0) become zeros.
cudaError_t int8_join_launch(const int32_t *part, int64_t ld_part, int64_t plane, int splits, const int32_t *row_group,
                             const float *x_scales, const float *scales, int64_t rows, int64_t cols, void *out,
                             int64_t ldo, int out_type, cudaStream_t s);

// Matrices at any pitch copied to one of a multiple of 16 bytes (those of groups that have rows).
cudaError_t int8_copy_launch(const int8_t *w, int64_t ldw, int64_t stride, int64_t rows, int64_t cols, int64_t batch,
                             int8_t *out, int64_t ldo, const int32_t *ends, cudaStream_t s);

}  // namespace sg
