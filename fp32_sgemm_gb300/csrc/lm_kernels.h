// What the host side of the language-model operators and their kernels share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace sg {

constexpr int kLmMaxGroups = 1024;
// Terms that one running sum of the tensor core may have: it truncates, so that
// terms of one sign lose up to 1.7e-7 of the sum for every 16 (f16; 9e-5 of it
// here, below a quarter of a unit in the last place of any 16-bit result).
constexpr int64_t kLmPlainTerms = 16384;
constexpr float kLog2E = 1.4426950408889634f;

// Wait / check site of the error word (bits 24..31) beside those of the
// main kernels: group ends that run backwards or past the last row.
constexpr uint32_t kSiteGroupEnds = 6;

enum LmRag { kRagNone = 0, kRagN = 1, kRagK = 2 };
enum LmEpi {
    kEpiCols = 0,      // D^T into a row-major matrix (columns of D are its rows)
    kEpiRows = 1,      // alpha * (D + acc_in) into a row-major matrix
    kEpiLse = 2,       // running maximum and sum of exponentials of each row of D
    kEpiDLogits = 3    // gradient of the loss by each element of D
};
enum LmOut { kOutF32 = 0, kOutF16 = 1, kOutBF16 = 2 };

struct LmArgs {
    int M, N;             // rows and columns of D (kRagN: columns by groups)
    int T;                // token rows (ragged extent)
    int kb;               // blocks of 64 of the contraction (not kRagK)
    int kb_plane;         // kRagNone: of one plane of A (kb, or half of it)
    int G;
    const int32_t *ends;  // [G] end row of each group
    int tiles_m, tiles_n, tile_n, num_tiles, splits, group_m;
    uint32_t bf16;        // operands bf16 (else f16)
    void *C;
    int64_t ldc, stride_c;   // stride_c: per group (kRagK) or per K split (FP32 partial sums)
    int out, vec;            // LmOut; vec: rows take aligned vector stores
    const float *acc_in;     // added to D before alpha, or NULL
    int64_t ld_acc;
    const float *alpha;      // device scalar, or NULL for 1
    // Loss epilogues; D's columns are vocabulary entries v0 .. v0 + N - 1.
    const int64_t *target;
    int64_t vocab, v0;
    float2 *part;            // [column slab][row] {maximum, sum}
    float *picked;           // logit of the row's target
    const float *lse, *grad, *gscale;
    void *lo;                // rest of the rounding to 16 bits, laid out as C, or NULL
    uint32_t *err;
    uint64_t timeout_ns;
    int withhold;
};

struct LmKernel {
    const void *fn = nullptr;
    int threads = 0, smem = 0, tile_m = 0, bn = 0, gran = 0, pair = 0, box_a = 0;
    int a_mn = 0;                   // A is read MN-major (boxes of 64 x 64)
};

// Operands of lm_rows32.cu as they lie in memory.
struct LmRows {
    const float *X, *W;
    int64_t ldx, ldw, stride;
    int K, x_vec, w_vec;            // rows take 16-byte loads
};
// tile_m columns by bn rows; few: fewer tiles than SMs.
LmKernel lm_rows32_kernel_info(bool trans, bool few);

// Kernel tables.  size: 0 thin, 1 middle, 2 big (SM pair); lengthy: 16-bit
// operands are summed in runs (see kLmPlainTerms).
LmKernel lm_grouped_kernel(int size, bool w_mn, bool f32, bool lengthy);      // lm_grouped*.cu
LmKernel lm_weight_grad_kernel(int size, bool f32, bool lengthy);             // size 1 or 2
LmKernel lm_lse_kernel(bool big, bool f32);                     // lm_loss*.cu
LmKernel lm_dlogits_kernel(bool big, bool f32);
LmKernel lm_rows_kernel(bool big, bool a_mn, bool f32, bool lengthy);         // B MN-major; MN-major A is big

// What of an operand a copy needs.  With targets: the rows whose target is an
// entry of the vocabulary and whose gradient is not zero, the others become
// zeros.  With ends: the matrices of a batch whose group has rows, the others
// are left as they are (no tile reads them).
struct LmCopyFilter {
    const int64_t *target = nullptr;
    int64_t vocab = 0;
    const float *grad = nullptr;
    const int32_t *ends = nullptr;
};

// lm_aux.cu.  An operand copy TMA can address: rows x cols (x batch) with
// pitch ld -> pitch ld_dst (a multiple of 8), 16-bit copied as they are, FP32
// as three bf16 planes (plane stride in elements).
struct LmCopy {
    const void *src = nullptr;       // NULL: nothing to copy
    int64_t ld = 0, stride = 0;
    void *dst = nullptr;
    int64_t ld_dst = 0, plane = 0, rows = 0, cols = 0, batch = 0;
    LmCopyFilter keep;
    int64_t chunks = 0, bytes = 0;   // chunks of 8 elements; from the first element to the last (set by the launch)
};
// scale2 = {top / m, m / top} for the largest |grad| m of a counted row.
struct LmGradScale {
    const float *grad = nullptr;
    const int64_t *target = nullptr;
    int64_t vocab = 0;
    int rows = 0;
    float top = 1.f;
    float *scale2 = nullptr;         // NULL: not wanted
};
// Both copies and the scale in one launch.
cudaError_t lm_launch_copy(bool f32, LmCopy a, LmCopy b, const LmGradScale &scale, cudaStream_t s);
// Joins the slabs' maxima and sums: lse and loss of each row.
cudaError_t lm_launch_lse_join(const float2 *part, int slabs, int rows, const float *picked, const int64_t *target,
                               int64_t vocab, float *loss, float *lse, cudaStream_t s);
// out = alpha * (sum of `splits` FP32 planes), rounded to `out_type`.
cudaError_t lm_launch_join_splits(const float *part, int64_t ld_part, int64_t plane, int splits, const float *alpha,
                                  int rows, int cols, void *out, int64_t ldo, int out_type, cudaStream_t s);
// rows x cols (x batch) elements of 2 or 4 bytes set to zero.
cudaError_t lm_launch_zero(void *p, int64_t ld, int64_t stride, int elem, int64_t rows, int64_t cols, int64_t batch,
                           cudaStream_t s);

}  // namespace sg
