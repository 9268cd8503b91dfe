/*
 * sgemm_norm.h -- layer norm over the rows of a matrix, and its gradients, in
 * single precision on gfx950.  Status codes are those of sgemm.h.
 *
 * The operation.  For each row x of N values,
 *
 *      mean = sum x / N,   rstd = 1 / sqrt(sum (x - mean)^2 / N + eps)
 *      y = (x - mean) rstd weight + bias
 *
 * where weight (1 without it) and bias (0 without it) have N values.
 *
 * Gradients.  With xh = (x - mean) rstd and g = dy weight,
 *
 *      dx      = rstd (g - mean(g) - xh mean(g xh)) + residual
 *      dweight = sum over rows of dy xh
 *      dbias   = sum over rows of dy
 *
 * residual is the gradient that reaches x by another way (the sum around a
 * layer), optional.
 *
 * Everything is summed in FP32: the mean first, then the squares of what is left
 * of it, which do not cancel however large the mean is.  The mean itself is an FP32
 * sum, rounded: it is off by a few 2^-24 of the row's mean |x|, and that times rstd
 * goes into every y of the row.  Squares past FP32 (|x - mean| over about 1e19) give
 * rstd = 0, a row whose sum is past FP32 gives NaN.  NaN and infinities give NaN in
 * their row, and in dweight and dbias of their columns.
 *
 * Contracts as for sgemm.h: device memory owned by the caller, 4-byte aligned,
 * any leading dimension; enqueued on stream without allocating or
 * synchronising; arguments checked before any HIP call; results the same from
 * run to run (no atomics).
 */
#ifndef SGEMM_NORM_H
#define SGEMM_NORM_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Y = layer norm of X's rows, both M x N.
 *   weight, bias  N floats, or NULL.
 *   eps           0 or more.
 *   Y             may be X itself (same pointer, ldx == ldy); otherwise it
 *                 does not overlap it.
 *   mean, rstd    out: M floats, or NULL; the gradients need both.
 * M == 0 or N == 0 is a no-op. */
int sgemm_layer_norm(int64_t M, int64_t N, const float *X, int64_t ldx,
                     const float *weight, const float *bias, float eps,
                     float *Y, int64_t ldy, float *mean, float *rstd,
                     hipStream_t stream);

/* The gradients for the gradient dY of Y; X, mean and rstd as above.
 *   weight        as above, or NULL.
 *   residual      M x N, added to dX, or NULL; row i at residual + i*ldr.
 *   dX            M x N, or NULL when only the sums are wanted.  May be dY,
 *                 X or residual itself (same pointer and leading dimension);
 *                 otherwise it overlaps none of them.
 *   dweight, dbias  N floats, or NULL.  0 where M == 0.
 *   workspace     room for the sums: sgemm_layer_norm_backward_workspace_bytes
 *                 bytes where dweight or dbias is wanted, 4-byte aligned; less
 *                 is SGEMM_ERR_INVALID_ARG.
 * N == 0 is a no-op. */
int sgemm_layer_norm_backward(int64_t M, int64_t N, const float *dY, int64_t lddy,
                              const float *X, int64_t ldx, const float *mean,
                              const float *rstd, const float *weight,
                              const float *residual, int64_t ldr, float *dX,
                              int64_t lddx, float *dweight, float *dbias,
                              hipStream_t stream, void *workspace,
                              int64_t workspace_bytes);
int64_t sgemm_layer_norm_backward_workspace_bytes(int64_t M, int64_t N);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_NORM_H */
