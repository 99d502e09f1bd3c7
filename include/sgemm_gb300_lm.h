/*
 * sgemm_gb300_lm.h: C ABI of the matrix products of language models on
 * NVIDIA GB300 (sm_103a), beside the FP32 product of sgemm_gb300.h:
 *
 *   - products grouped by expert with ragged group sizes, and their
 *     gradients (sgemmGrouped, sgemmGroupedWeightGrad);
 *   - softmax cross entropy over a vocabulary whose logits are never kept,
 *     and its gradients (sgemmCrossEntropy, sgemmCrossEntropyGrad);
 *   - products of a few rows with 4-bit weights and group scales
 *     (sgemmW4);
 *   - products in 8-bit integers with scales for each token and channel, by
 *     expert or not (sgemmInt8, sgemmInt8Quantize);
 *   - a router's choice of experts and its gradient (sgemmRouteTopK), tokens
 *     sorted by expert and brought back, and their gradients
 *     (sgemmExpertDispatch, sgemmExpertCombine).
 *
 * The conventions of sgemm_gb300.h hold: row-major matrices with explicit
 * row pitches in elements, device pointers, work only enqueued on `stream`,
 * no allocation, a handle per stream, the workspace attached with
 * sgemmSetWorkspace(), errors returned.  Pointers are aligned to their
 * element type; operands that TMA cannot address (base not 16-byte aligned
 * or pitch not a multiple of 16 bytes) are copied into the workspace first.
 * Sums are FP32 in every type (of 8-bit integers: exact); each result is rounded
 * once to its type.
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
    SGEMM_TYPE_BF16 = 2,
    SGEMM_TYPE_S8 = 3           /* the rows of sgemmInt8() alone */
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
 * F16 and BF16 products run on the tensor cores with FP32 sums, in runs of 8192
 * terms where the contraction may have more than 16384 (the tensor cores' sums
 * truncate: by up to 1.7e-7 of the sum for every 16 terms of one sign).  F32
 * products of up to 8 rows a group in the mean (T / G) and K >= 256 are
 * FP32 multiply-adds.  For the others F32 operands are split into three bf16
 * planes each in the workspace (x = p0 + p1 + p2, each plane the nearest to
 * what is left; exact for |x| >= 2^-110) and multiplied as the six products
 * p_i q_j, i + j <= 2, with FP32 sums of 64-long pieces; the plane products
 * left out are below 2^-23 of a product, with either sign (2^-22 if a factor
 * is above 3.38e38).  There infinite F32 inputs give NaN or infinity.
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

/* Workspace sgemmGrouped() requires: copies of operands that are not read in
   place, partial sums where few rows leave the contraction to be cut. */
sgemmStatus_t sgemmGroupedWorkspaceSize(sgemmHandle_t handle, sgemmDataType_t type, sgemmOperation_t opB, int64_t T,
                                        int64_t N, int64_t K, int64_t G, const void *A, int64_t lda, const void *B,
                                        int64_t ldb, int64_t strideB, size_t *bytes);

/* What sgemmGrouped() or sgemmGroupedWeightGrad() runs for a call of these
   sizes (nothing is launched). */
typedef struct sgemmGroupedPlan {
    int kernel;             /* 0 none (an empty product), 1 FP32 multiply-adds, 2 tensor cores, a tile per SM,
                               3 tensor cores, a tile per pair of SMs */
    int tile_m, tile_n;     /* rows and columns of C_g in one tile, at most */
    int splits;             /* parts the contraction is cut into */
    int copies_a, copies_b; /* 1 if the operand is copied into the workspace */
} sgemmGroupedPlan_t;

sgemmStatus_t sgemmGroupedQueryPlan(sgemmHandle_t handle, sgemmDataType_t type, sgemmOperation_t opB, int64_t T,
                                    int64_t N, int64_t K, int64_t G, const void *A, int64_t lda, const void *B,
                                    int64_t ldb, int64_t strideB, sgemmGroupedPlan_t *plan);

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

sgemmStatus_t sgemmGroupedWeightGradQueryPlan(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t M,
                                              int64_t N, int64_t G, const void *A, int64_t lda, const void *B,
                                              int64_t ldb, sgemmGroupedPlan_t *plan);

/*
 * Softmax cross entropy over a vocabulary.  X is T x D (one row per token),
 * W is V x D (one row per vocabulary entry), target[t] a vocabulary index:
 *
 *   lse[t]  = log sum_v exp(X[t, :] . W[v, :])
 *   loss[t] = lse[t] - X[t, :] . W[target[t], :]
 *
 * The T x V logits are never written to memory: each tile of them is
 * reduced to a maximum and a sum of exponentials per row where it was
 * computed, and the partial results are joined in a fixed order.  A target
 * outside [0, V) marks a token that is not counted: its loss is 0 (its lse
 * is computed).  loss and lse are FP32 in every type.  Arithmetic of the
 * products as for sgemmGrouped(), 16-bit ones here in sums of 512 terms of
 * the contraction, added in FP32.  INVALID_VALUE also for V < 1 or D < 1;
 * T == 0 is a no-op.  A workspace is always required (the partial results).
 */
sgemmStatus_t sgemmCrossEntropy(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t V, int64_t D,
                                const void *X, int64_t ldx, const void *W, int64_t ldw, const int64_t *target,
                                float *loss, float *lse, cudaStream_t stream);

sgemmStatus_t sgemmCrossEntropyWorkspaceSize(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t V,
                                             int64_t D, const void *X, int64_t ldx, const void *W, int64_t ldw,
                                             size_t *bytes);

/*
 * Its gradients, from the lse of sgemmCrossEntropy() and the gradient
 * dloss[t] (FP32) by each token's loss:
 *
 *   d[t, v] = dloss[t] * (exp(X[t, :] . W[v, :] - lse[t]) - [v == target[t]])
 *   dX = d . W        dW = d^T . X
 *
 * The logits are summed as in sgemmCrossEntropy(), so that a row's
 * probabilities add up to one.  The vocabulary is taken in pieces: d is
 * computed for one piece at a time (512 MB at most, or 2048 columns) and both
 * products over the piece follow; dX is summed over the pieces in FP32.  How d
 * is held:
 *   F32              FP32, then three bf16 planes;
 *   up to 128 rows   two planes of the call's type, d and what its rounding
 *                    left (16 bits and more of significand);
 *   more rows        one plane of the call's type.
 * F16 in either, and BF16 in one plane, hold d divided by the largest
 * |dloss| of a counted token (F16: times 2^13 besides, above f16's subnormal
 * numbers), taken in again in FP32 by the products.  (Where that largest is
 * outside [1e-30, 1e30], d is held as it is.)
 *
 * Tokens that are not counted, and those with dloss 0, have no part in
 * either gradient whatever their rows of X hold, infinities and NaN too (X
 * is always copied into the workspace, with zeros in their place); their dX
 * is zero.  T == 0 sets dW to zero.
 */
sgemmStatus_t sgemmCrossEntropyGrad(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t V, int64_t D,
                                    const void *X, int64_t ldx, const void *W, int64_t ldw, const int64_t *target,
                                    const float *lse, const float *dloss, void *dX, int64_t lddx, void *dW,
                                    int64_t lddw, cudaStream_t stream);

sgemmStatus_t sgemmCrossEntropyGradWorkspaceSize(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t V,
                                                 int64_t D, const void *X, int64_t ldx, const void *W, int64_t ldw,
                                                 size_t *bytes);

/*
 * Products of a few rows with 4-bit weights and group scales.  X is M x K,
 * the weights are N x K (one row per output column), two to a byte along K:
 * Q is N rows of K / 2 bytes (pitch ldq BYTES), column 2 i in the low four
 * bits of byte i, column 2 i + 1 in the high four.  Each row has a scale (of
 * the call's type; pitch lds) and, if `zeros` is not NULL, a zero point (any
 * byte, 0 to 255; pitch ldz; otherwise 8) for every `group` columns:
 *
 *   Y[t, n] = sum_k scales[n, k / group] * (q[n, k] - zeros[n, k / group]) * X[t, k]
 *
 * group is 32, 64 or 128 and divides K.  q - zero meets X unrounded and
 * unscaled, the scale is applied to each group's FP32 sum; F32 X is split
 * into three bf16 planes (exactly for |x| >= 2^-110).  One pass over the weights serves up to
 * 32 rows (F32: 10); more rows take further passes.
 *
 * INVALID_VALUE, NOT_SUPPORTED as above, also for another group or a K it
 * does not divide.  MISALIGNED also when Q is not 16-byte aligned or ldq not
 * a multiple of 16 bytes.  WORKSPACE_REQUIRED when X is too long for shared
 * memory and K is cut (the size query says).  M == 0 or N == 0 is a no-op;
 * K == 0 sets Y to zero.
 */
sgemmStatus_t sgemmW4(sgemmHandle_t handle, sgemmDataType_t type, int64_t M, int64_t N, int64_t K, int group,
                      const void *X, int64_t ldx, const uint8_t *Q, int64_t ldq, const void *scales, int64_t lds,
                      const uint8_t *zeros, int64_t ldz, void *Y, int64_t ldy, cudaStream_t stream);

sgemmStatus_t sgemmW4WorkspaceSize(sgemmHandle_t handle, sgemmDataType_t type, int64_t M, int64_t N, int64_t K,
                                   int group, size_t *bytes);

/*
 * Rows as 8-bit integers with a scale each: X is T x K,
 *
 *   scales[t] = max_k |X[t, k]| / 127      (the nearest FP32 number, at least 2^-126; 0 for a row of zeros)
 *   Q[t, k]   = X[t, k] / scales[t] rounded to the nearest integer, ties to even
 *
 * (pitch ldq BYTES; the bytes between K and the pitch are not written.)  A row
 * with an infinity or a NaN has scale NaN and integers 0, so that its products
 * are NaN.  T == 0 is a no-op.
 */
sgemmStatus_t sgemmInt8Quantize(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t K, const void *X,
                                int64_t ldx, int8_t *Q, int64_t ldq, float *scales, cudaStream_t stream);

/*
 * Products in 8-bit integers.  The weights are N x K integers (one row per
 * output column, pitch ldb BYTES) with a scale for each row; with G > 1 or
 * groupEnds there is one such matrix per group, at B + g * strideB, its scales
 * at scales + g * N, and the rows of X are sorted by group as for
 * sgemmGrouped().  groupEnds may be NULL if G == 1: then all rows have the one
 * matrix.  X is T x K, of integers (SGEMM_TYPE_S8, pitch ldx BYTES) with their
 * scales xScales[t], or of a type of numbers: then xScales is NULL and each row
 * becomes integers as by sgemmInt8Quantize().
 *
 *   C[t, n] = xScales[t] * scales[g, n] * sum_k X[t, k] B_g[n, k]
 *
 * The sum is exact (a 32-bit integer); it becomes FP32, is multiplied by the
 * row's scale, then by the channel's, and is rounded to typeC: the same bits
 * whatever the number of rows, the groups or the pitches.  Rows behind the last
 * end become zeros; ends that run backwards are treated as in sgemmGrouped().
 *
 * INVALID_VALUE, MISALIGNED, NOT_SUPPORTED as for sgemmGrouped(), also for
 * xScales that is NULL with integers or not NULL with numbers; NOT_SUPPORTED for
 * K > 131071, beyond which a sum may pass 32 bits.  W that is not 16-byte aligned
 * with pitches that are multiples of 16 is read more slowly, or copied.
 * WORKSPACE_REQUIRED: see the size query.  T == 0 or N == 0 is a no-op; K == 0 or
 * G == 0 sets C to zero.
 */
sgemmStatus_t sgemmInt8(sgemmHandle_t handle, sgemmDataType_t typeX, sgemmDataType_t typeC, int64_t T, int64_t N,
                        int64_t K, int64_t G, const void *X, int64_t ldx, const float *xScales, const int8_t *B,
                        int64_t ldb, int64_t strideB, const float *scales, const int32_t *groupEnds, void *C,
                        int64_t ldc, cudaStream_t stream);

sgemmStatus_t sgemmInt8WorkspaceSize(sgemmHandle_t handle, sgemmDataType_t typeX, sgemmDataType_t typeC, int64_t T,
                                     int64_t N, int64_t K, int64_t G, const void *X, int64_t ldx, const int8_t *B,
                                     int64_t ldb, int64_t strideB, size_t *bytes);

/*
 * A router's choice.  Each of T tokens has E logits (pitch ldl); the k largest
 * are chosen, in falling order, the lower index first among equals (0 and -0
 * are equal; NaN counts as larger than every number).  With
 * p = softmax(logits[t, :]):
 *
 *   experts[t * k + j] = e_j
 *   weights[t * k + j] = p[e_j]                            normalize == 0
 *                      = p[e_j] / sum_i p[e_i]             otherwise
 *
 * A logit of -inf is an expert that is masked: it is never chosen, and where
 * fewer than k are left the remaining choices are -1 with weight 0.  (The lowest
 * finite value of a type is a number like any other.)  A NaN or +inf among a
 * token's logits makes its weights NaN.  Weights and sums are FP32 in every type.
 *
 * The gradient by the logits from that by the weights, for the same choice,
 * S being the experts chosen (-1 and what lies outside [0, E) take no part):
 *
 *   dlogits[t, e] = p_e ([e in S] dweights_e - sum_S p_i dweights_i)
 *
 * with the normalized weights in the place of p, and 0 outside S, if normalize.
 *
 * INVALID_VALUE: negative T, E < 1, k < 1, k > E, NULL pointers with nonzero
 * extent, and as for sgemmGrouped().  NOT_SUPPORTED: E > 1024, k > 32, T * k of
 * 2^31 or more.  T == 0 is a no-op.  No workspace.
 */
sgemmStatus_t sgemmRouteTopK(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t E, int64_t k,
                             int normalize, const void *logits, int64_t ldl, float *weights, int64_t *experts,
                             cudaStream_t stream);

sgemmStatus_t sgemmRouteTopKGrad(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t E, int64_t k,
                                 int normalize, const void *logits, int64_t ldl, const int64_t *experts,
                                 const float *dweights, void *dlogits, int64_t ldd, cudaStream_t stream);

/*
 * Tokens sorted by expert: X is T x D, experts T x k (any number outside
 * [0, G) is no expert; a token may choose an expert more than once).  The T * k
 * choices are sorted by expert, each expert's in their order in `experts`, and
 *
 *   rows[slots[t, j], :] = X[t, :]
 *   groupEnds[g] = the row at which expert g's rows end     (as sgemmGrouped() takes them)
 *
 * Choices of no expert come behind the last end: their row r holds zeros and
 * is written as ~r (that is -1 - r) in slots, which so names each of the T * k
 * rows once.  rows is (T * k) x D.  The gradient by X is
 * sgemmExpertCombine() of the rows' gradient without weights.
 *
 * Back again, with FP32 weights [T, k] (NULL: 1):
 *
 *   Y[t, :] = sum_j weights[t, j] * rows[slots[t, j], :]     over slots[t, j] in [0, T * k)
 *
 * in the order of j, in FP32, rounded once.  Its gradients, either of which
 * may be NULL:
 *
 *   dRows[slots[t, j], :] = weights[t, j] * dY[t, :]
 *   dRows[r, :] = 0                                           for a row r that no slot names
 *   dWeights[t, j] = dY[t, :] . rows[slots[t, j], :]          (0 for a slot that names no row)
 *
 * A negative slot, or one of T * k or more, names no row, and a row is named at
 * most once (of one named twice dRows is undefined).  Which rows no slot
 * names is noted in `owners`, T * k numbers of scratch.  Without them (NULL, or
 * sgemmExpertCombineGrad()) the slots have to be those of sgemmExpertDispatch():
 * row ~slots[t, j] of a negative slot gets zeros, and a row that is named neither
 * way keeps what was there.
 *
 * INVALID_VALUE, MISALIGNED as for sgemmGrouped().  NOT_SUPPORTED: T * k, D of
 * 2^31 or more, G > SGEMM_MAX_GROUPS.  No workspace.
 */
sgemmStatus_t sgemmExpertDispatch(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t D, int64_t k,
                                  int64_t G, const void *X, int64_t ldx, const int64_t *experts, void *rows,
                                  int64_t ldr, int32_t *slots, int32_t *groupEnds, cudaStream_t stream);

sgemmStatus_t sgemmExpertCombine(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t D, int64_t k,
                                 const void *rows, int64_t ldr, const int32_t *slots, const float *weights, void *Y,
                                 int64_t ldy, cudaStream_t stream);

sgemmStatus_t sgemmExpertCombineGrad(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t D, int64_t k,
                                     const void *dY, int64_t lddy, const void *rows, int64_t ldr,
                                     const int32_t *slots, const float *weights, void *dRows, int64_t lddr,
                                     float *dWeights, cudaStream_t stream);

sgemmStatus_t sgemmExpertCombineGradEx(sgemmHandle_t handle, sgemmDataType_t type, int64_t T, int64_t D, int64_t k,
                                       const void *dY, int64_t lddy, const void *rows, int64_t ldr,
                                       const int32_t *slots, const float *weights, void *dRows, int64_t lddr,
                                       float *dWeights, int32_t *owners, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_GB300_LM_H */
