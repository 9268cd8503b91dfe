/*
 * sgemm_xent.h -- softmax cross entropy of a product's rows, and its gradients,
 * in single precision on gfx950, without the product in memory.  Status codes are
 * those of sgemm.h.
 *
 * The operation.  T rows of H values are scored against a vocabulary of V,
 *
 *      Z = X·op(B)          T x V; op(B) is B (H x V) or, with trans_b, the
 *                           transpose of a stored V x H matrix
 *      lse[t]  = log(sum over v of exp(Z[t][v]))
 *      loss[t] = lse[t] - Z[t][targets[t]]
 *
 * A row whose target is outside 0 .. V-1 (-1 or -100, say) has none: its loss and
 * lse are 0, and it reaches no gradient, whatever its X and dloss hold, NaN
 * included.
 *
 * Gradients.  With dloss[t] the gradient of loss[t],
 *
 *      dZ[t][v] = (exp(Z[t][v] - lse[t]) - [v == targets[t]]) dloss[t]
 *      dX = dZ·op(B)^T,   d op(B) = X^T·dZ
 *
 * Z and dZ are never whole in memory: forward, each tile of Z leaves a row's
 * largest value and sum of exponentials; backward, Z is made again and dZ kept a
 * piece of the vocabulary at a time.  Rows without a target are left out of the
 * products; which ones they are stays on the device.
 *
 * Contracts as for sgemm.h and sgemm_linear.h: device memory owned by the caller,
 * 4-byte aligned (targets of 8 bytes 8-byte aligned); enqueued on stream without
 * allocating or synchronising; arguments checked before any HIP call; results the
 * same from run to run (no atomics).  Leading dimensions of X and B, V and H are
 * limited to SGEMM_XENT_MAX_LD; more is SGEMM_ERR_UNSUPPORTED.  Infinite and NaN
 * logits follow the formulas: a row with one of +infinity has lse = +infinity and a dZ
 * that is NaN there alone, one with a NaN has NaN.  Finite ones are taken to be below
 * 2e38 in size.
 */
#ifndef SGEMM_XENT_H
#define SGEMM_XENT_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SGEMM_XENT_MAX_LD (1 << 20)

/* loss and lse of every row.
 *   trans_b    0 or 1.
 *   X, ldx     T x H, ldx >= max(1, H).
 *   B, ldb     H x V, ldb >= max(1, V); with trans_b V x H, ldb >= max(1, H).
 *   targets    T ids, id_bytes 4 (int32) or 8 (int64) bytes each.
 *   loss       out: T floats.
 *   lse        out: T floats, or NULL; the gradients need it.
 *   workspace  sgemm_linear_xent_workspace_bytes bytes, 4-byte aligned; less is
 *              SGEMM_ERR_INVALID_ARG.
 * T == 0 is a no-op. */
int sgemm_linear_xent(int trans_b, int64_t T, int64_t V, int64_t H,
                      const float *X, int64_t ldx, const float *B, int64_t ldb,
                      const void *targets, int id_bytes, float *loss, float *lse,
                      hipStream_t stream, void *workspace, int64_t workspace_bytes);
int64_t sgemm_linear_xent_workspace_bytes(int trans_b, int64_t T, int64_t V, int64_t H);

/* dX (T x H, rows without a target 0) and dB (stored like B) for dloss and the lse
 * that sgemm_linear_xent gave.
 *   dX, lddx   or NULL when only dB is wanted.
 *   dB, lddb   or NULL when only dX is wanted.
 *   dX and dB overlap no operand.
 *   workspace  4-byte aligned.  sgemm_linear_xent_backward_workspace_bytes is what
 *              the fastest plan takes (a larger one changes nothing); with less the
 *              vocabulary goes in more pieces, down to
 *              sgemm_linear_xent_backward_least_bytes, below which it is
 *              SGEMM_ERR_INVALID_ARG.
 * T == 0 sets dB to 0; H == 0 or V == 0 leaves nothing but dX = 0.  T H (H in fours)
 * of 2^34 or more is SGEMM_ERR_UNSUPPORTED. */
int sgemm_linear_xent_backward(int trans_b, int64_t T, int64_t V, int64_t H,
                               const float *X, int64_t ldx, const float *B,
                               int64_t ldb, const void *targets, int id_bytes,
                               const float *lse, const float *dloss, float *dX,
                               int64_t lddx, float *dB, int64_t lddb,
                               hipStream_t stream, void *workspace,
                               int64_t workspace_bytes);
int64_t sgemm_linear_xent_backward_workspace_bytes(int trans_b, int64_t T, int64_t V,
                                                   int64_t H);
int64_t sgemm_linear_xent_backward_least_bytes(int trans_b, int64_t T, int64_t V,
                                               int64_t H);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_XENT_H */
