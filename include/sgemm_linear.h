/*
 * sgemm_linear.h -- products with an epilogue, and their gradients, in single
 * precision on gfx950.  Status codes are those of sgemm.h.
 *
 * The operation.  With op(A) of M x K and op(B) of K x N,
 *
 *      Z = op(A)·op(B) + bias          (bias: N values, added to every row)
 *      C = act(Z) + residual           (residual: M x N)
 *
 * where bias, act and residual are each optional and Z can be stored as well
 * (it is what the gradient of act needs).  Storage is row-major with leading
 * dimensions, as in sgemm.h; op(A) is A (M x K) or, with trans_a, the
 * transpose of a stored K x M matrix, and op(B) is B (K x N) or, with
 * trans_b, the transpose of a stored N x K matrix (a layer's weight kept
 * "out x in").  The products accumulate in FP32 and everything of the
 * epilogue is computed in FP32.
 *
 * Gradients.  With dC the gradient of C:
 *
 *      dZ        = dC * act'(Z)        sgemm_act_backward
 *      dbias     = sum over rows of dZ sgemm_act_backward
 *      dresidual = dC
 *      d op(A)   = dZ·op(B)^T          sgemm_linear, trans_b flipped
 *      d op(B)   = op(A)^T·dZ          sgemm_linear, trans_a flipped
 *
 * Activations, with Phi the normal distribution function:
 *      NONE z;  RELU max(z, 0);  GELU z Phi(z);  SILU z / (1 + exp(-z));
 *      GELU_TANH z / (1 + exp(-2u)), u = sqrt(2/pi) (z + 0.044715 z^3),
 *      which is z (1 + tanh u) / 2.
 * RELU's derivative at 0 is 0.  NaN gives NaN; at +-inf the activations and
 * their derivatives take their limits.
 *
 * Contracts as for sgemm.h unless said otherwise: device memory owned by the
 * caller, 4-byte aligned, any leading dimension; enqueued on stream without
 * allocating or synchronising; arguments checked before any HIP call; results
 * the same from run to run (no atomics).
 */
#ifndef SGEMM_LINEAR_H
#define SGEMM_LINEAR_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SGEMM_ACT_NONE 0
#define SGEMM_ACT_RELU 1
#define SGEMM_ACT_GELU 2
#define SGEMM_ACT_GELU_TANH 3
#define SGEMM_ACT_SILU 4

/* The epilogue of a product; a NULL sgemm_epilogue is all zeros. */
typedef struct sgemm_epilogue {
    int act;                /* SGEMM_ACT_* */
    const float *bias;      /* N floats, or NULL.  sgemm_grouped: N floats
                               for each group, group g's at bias + g*ldbias */
    int64_t ldbias;         /* sgemm_grouped only: >= max(1, N) */
    const float *residual;  /* M x N, or NULL; row i at residual + i*ldr */
    int64_t ldr;
    float *preact;          /* out: Z, M x N, or NULL; row i at preact + i*ldp */
    int64_t ldp;
} sgemm_epilogue;

/* C (and epilogue->preact) as above.
 *   trans_a, trans_b  0 or 1.
 *   A, lda   M x K, lda >= max(1, K); with trans_a K x M, lda >= max(1, M).
 *   B, ldb   K x N, ldb >= max(1, N); with trans_b N x K, ldb >= max(1, K).
 *   C, ldc   M x N, ldc >= max(1, N); not overlapping A, B, bias or preact.
 *            residual may be C itself (same pointer, ldr == ldc: added in
 *            place) or must not overlap it.  preact overlaps nothing.
 *   workspace, workspace_bytes   as for sgemm_ws: room for K to be split
 *            across workgroups where that is faster; 0 allows no split.
 *            sgemm_linear_workspace_bytes tells what the fastest plan wants;
 *            a larger one changes nothing.
 * K == 0 gives Z = bias (or 0); M == 0 or N == 0 is a no-op.  Errors as for
 * sgemm and sgemm_ws, an unknown act or a bad epilogue leading dimension or
 * pointer being SGEMM_ERR_INVALID_ARG. */
int sgemm_linear(int trans_a, int trans_b, int64_t M, int64_t N, int64_t K,
                 const float *A, int64_t lda, const float *B, int64_t ldb,
                 float *C, int64_t ldc, const sgemm_epilogue *epilogue,
                 hipStream_t stream, void *workspace, int64_t workspace_bytes);

/* The workspace sgemm_linear takes for its fastest plan (0: none).  Host
 * only. */
int64_t sgemm_linear_workspace_bytes(int trans_a, int trans_b, int64_t M,
                                     int64_t N, int64_t K);

/* What sgemm_linear would launch for contiguous operands aligned to 16 bytes
 * and this much workspace.  A kernel "product_.." is a tile of matrix
 * instructions (then 's' or 'f' for A and B: k from row to row or along the
 * rows), "rows_.." the vector kernels for a few rows, for which tile_k,
 * lds_bytes and wg_per_cu are 0.  A product a little over whole rounds of its
 * tiles is cut in two launches: "+4rows" or "+4cols" is what the second one
 * computes, the plan is the first one's but for workspace_bytes, which is
 * enough for both.  Host only. */
int sgemm_linear_plan_query(int trans_a, int trans_b, int64_t M, int64_t N,
                            int64_t K, int64_t workspace_bytes,
                            sgemm_plan *plan);

/* dZ = dC * act'(preact) and dbias[j] = sum_i dZ[i][j], for M x N matrices.
 *   preact    Z as sgemm_linear stored it; not read (may be NULL) for
 *             SGEMM_ACT_NONE.
 *   dZ        M x N, or NULL when only dbias is wanted.  May be dC itself
 *             (same pointer, lddz == lddc) or preact itself; otherwise it
 *             overlaps neither.
 *   dbias     N floats, or NULL.  With M == 0 it is set to 0.
 *   workspace as above: room for the partial sums of dbias,
 *             sgemm_act_backward_workspace_bytes; with less the sums are a
 *             pass of their own over dZ, slower, with the same result. */
int sgemm_act_backward(int64_t M, int64_t N, const float *dC, int64_t lddc,
                       const float *preact, int64_t ldp, int act, float *dZ,
                       int64_t lddz, float *dbias, hipStream_t stream,
                       void *workspace, int64_t workspace_bytes);
int64_t sgemm_act_backward_workspace_bytes(int64_t M, int64_t N);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_LINEAR_H */
