/*
 * sgemm_gb300_lm.h: C ABI of the matrix products of language models on
 * NVIDIA GB300 (sm_103a), beside the FP32 product of sgemm_gb300.h:
 *
 *   - products grouped by expert with ragged group sizes, and their
 *     gradients (sgemmGrouped, sgemmGroupedWeightGrad);
 *   - softmax cross entropy over a vocabulary whose logits are never kept,
 *     and its gradients (sgemmCrossEntropy, sgemmCrossEntropyGrad);
 *   - products of a few rows with 4-bit weights and group scales
 *     (sgemmW4).
 *
 * The conventions of sgemm_gb300.h hold: row-major matrices with explicit
 * row pitches in elements, device pointers, work only enqueued on `stream`,
 * no allocation, a handle per stream, the workspace attached with
 * sgemmSetWorkspace(), errors returned.  Pointers are aligned to their
 * element type; operands that TMA cannot address (base not 16-byte aligned
 * or pitch not a multiple of 16 bytes) are copied into the workspace first.
 * Sums are FP32 in every type; each result is rounded once to its type.
 * Results are the same bits for the same call.  Outputs may not overlap
 * inputs.  Calls can be captured in CUDA graphs under the conditions of
 * sgemm_gb300.h.
 */
#ifndef SGEMM_GB300_LM_H
#define SGEMM_GB300_LM_H

#include "sgemm_gb300.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of the matrices of a call. */
typedef enum sgemmDataType {
    SGEMM_TYPE_F32 = 0,
    SGEMM_TYPE_F16 = 1,
    SGEMM_TYPE_BF16 = 2
} sgemmDataType_t;

/* Most groups of one call. */
#define SGEMM_MAX_GROUPS 1024

/*
 * Products grouped by expert.  A is T x K; its rows are sorted by group:
 * group g holds rows [groupEnds[g-1], groupEnds[g]) (from row 0 for g = 0),
 * groupEnds being G increasing row numbers IN DEVICE MEMORY, so that a
 * router's counts never visit the host.  Group g has a matrix B_g at
 * B + g * strideB: K x N (opB == SGEMM_OP_N, ldb >= N) or N x K
 * (SGEMM_OP_T, ldb >= K).
 *
 *   C[t, :] = A[t, :] . op(B_g)     for every row t of group g
 *
 * A group may be empty.  Rows behind the last end belong to no group: they
 * are set to zero (their A is not used).  Ends that run backwards or lie outside [0, T]
 * are pulled into range, recorded in the handle's error word (site 6 of
 * sgemmGetDeviceError; C is then undefined but nothing outside it is
 * touched).  The gradient by the rows is the same call with the output's
 * gradient as A and the other opB.
 *
 * F16 and BF16 products run on the tensor cores with FP32 sums.  F32
 * operands are split into three bf16 planes each (x = p0 + p1 + p2 exactly)
 * in the workspace and multiplied as the six products p_i q_j, i + j <= 2,
 * with FP32 sums of 64-long pieces; the planes left out are below 2^-23 of
 * a product.  Infinite F32 inputs give NaN or infinity.
 *
 * INVALID_VALUE: negative sizes, a pitch below the row length, strideB
 * below one matrix when G > 1, unknown type or op, NULL pointers with
 * nonzero extent, a NULL handle, another current device than the handle's.
 * MISALIGNED: a pointer not aligned to its element.  NOT_SUPPORTED: an
 * extent of 2^31 or more, G > SGEMM_MAX_GROUPS, an operand of 2^40 bytes.
 * WORKSPACE_REQUIRED: see the size query.  T == 0 or N == 0 is a no-op;
 * K == 0 or G == 0 sets C to zero.
 */
sgemmStatus_t sgemmGrouped(sgemmHandle_t handle, sgemmDataType_t type, sgemmOperation_t opB, int64_t T, int64_t N,
                           int64_t K, int64_t G, const void *A, int64_t lda, const void *B, int64_t ldb,
                           int64_t strideB, const int32_t *groupEnds, void *C, int64_t ldc, cudaStream_t stream);

/* Workspace sgemmGrouped() requires (0 for 16-bit operands read in place). */
sgemmStatus_t sgemmGroupedWorkspaceSize(sgemmHandle_t handle, sgemmDataType_t type, sgemmOperation_t opB, int64_t T,
                                        int64_t N, int64_t K, int64_t G, const void *A, int64_t lda, const void *B,
                                        int64_t ldb, int64_t strideB, size_t *bytes);

/*
 * Gradient by the groups' matrices: A is T x M, B is T x N, rows sorted by
 * group as for sgemmGrouped(),
 *
 *   C_g = A[rows of g, :]^T . B[rows of g, :]      (M x N, at C + g * strideC)
 *
 * zero for an empty group.  Rows behind the last end take no part, whatever
 * they hold.  With A the rows and B the output's gradient this is the
 * gradient of K x N matrices (opB == SGEMM_OP_N above); with the two
 * exchanged, that of N x K ones.  Types, arithmetic and errors as above;
 * M == 0, N == 0 or G == 0 is a no-op.
 */
sgemmStatus_t sgemmGroupedWeightGrad(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t M, int64_t N,
                                     int64_t G, const void *A, int64_t lda, const void *B, int64_t ldb,
                                     const int32_t *groupEnds, void *C, int64_t ldc, int64_t strideC,
                                     cudaStream_t stream);

sgemmStatus_t sgemmGroupedWeightGradWorkspaceSize(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t M,
                                                  int64_t N, int64_t G, const void *A, int64_t lda, const void *B,
                                                  int64_t ldb, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GB300_LM_H */
