/*
 * sgemm_moe.h -- mixture-of-experts routing and the experts' products, in
 * single precision on gfx950.  Status codes are those of sgemm.h, epilogue
 * and activations those of sgemm_linear.h.
 *
 * The path.  T tokens choose `top` of E experts each, which makes T·top rows:
 *
 *      sgemm_moe_route      a router's logits -> choices and their weights
 *      sgemm_moe_sort       choices -> offsets, order, place
 *      sgemm_moe_permute    each token's row to its places, in expert order
 *      sgemm_grouped        expert e's product over rows offsets[e] ..
 *                           offsets[e+1]-1
 *      sgemm_moe_unpermute  each token's rows back, weighted and summed
 *
 * A choice outside 0..E-1 (-1, say) is dropped: it has no row.  The kept rows
 * are numbered 0 .. offsets[E]-1; rows from offsets[E] on are neither read
 * nor written by any call here.  How many rows an expert has stays on the
 * device: no call waits for it.
 *
 * Gradients:
 *      permute    dX[t] = sum over t's rows of dXp: sgemm_moe_unpermute
 *                 without weights
 *      unpermute  sgemm_moe_unpermute_backward
 *      route      sgemm_moe_route_backward
 *      grouped    dZ and dbias: sgemm_grouped_act_backward; dA: sgemm_grouped
 *                 with trans_b flipped; dB: sgemm_grouped_wgrad
 *
 * Contracts (ownership, ordering, alignment, errors, determinism) as for
 * sgemm_linear.h.  Index arrays are device memory, int32, 4-byte aligned.
 * Their contents cannot be checked before a launch, and a bad value never
 * makes a kernel leave its operands: offsets are clamped to 0 .. rows, and a
 * place outside 0 .. T·top-1 counts as dropped.
 */
#ifndef SGEMM_MOE_H
#define SGEMM_MOE_H

#include "sgemm_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SGEMM_MOE_MAX_EXPERTS 1024
#define SGEMM_MOE_MAX_TOP 32       /* sgemm_moe_route's choices a token */
#define SGEMM_MOE_MAX_GROUPS 32    /* and groups of experts */

#define SGEMM_SCORE_SOFTMAX 0
#define SGEMM_SCORE_SIGMOID 1

/* How a router chooses.  With l a token's E logits:
 *
 *      s = softmax(l), or 1 / (1 + exp(-l)) for each expert
 *      c = s + bias       (the bias balances the choice, the weights are of s)
 *
 * With groups > 1 the experts are `groups` equal groups of neighbours; a group's
 * score is its best c, or with group_best 2 the sum of its best two (of the best
 * one where only one can be chosen), and the experts outside the best
 * `top_groups` groups cannot be chosen.  The best `top` c's are the choices, the
 * best first; equal scores go to the lowest expert (group).  The weights are s of
 * the choices, divided by their sum with renormalize, times scale. */
typedef struct sgemm_moe_router {
    int scoring;            /* SGEMM_SCORE_* */
    int renormalize;        /* 0 or 1 */
    float scale;            /* finite, not 0 */
    const float *bias;      /* E floats, or NULL */
    int groups;             /* 1 .. SGEMM_MOE_MAX_GROUPS, dividing E */
    int top_groups;         /* 1 .. groups */
    int group_best;         /* 1 or 2, at most E / groups */
} sgemm_moe_router;

/* experts and weights (T x top, contiguous) from logits (T x E, leading dimension
 * ldl).
 *   top   1 .. SGEMM_MOE_MAX_TOP, at most the experts of top_groups groups.
 * An expert whose logit or whose c is -infinity is never chosen: where fewer than
 * top remain, the rest of a token's choices are -1 with weight 0, which
 * sgemm_moe_sort drops.  A NaN score counts as infinite, and makes NaN weights.
 * The choice is that of the scores in FP64: what FP32 cannot tell apart is computed
 * again, and only what FP64 rounds to the same number is equal (two sigmoids next to
 * 1 with a bias, say).  Without a bias, and without groups of two scores, the logits
 * themselves decide, whose order is that of exact scores.  Experts over SGEMM_MOE_MAX_EXPERTS, top or groups over
 * their limits are SGEMM_ERR_UNSUPPORTED.  T == 0 is a no-op. */
int sgemm_moe_route(int64_t T, int64_t E, int64_t top, const float *logits,
                    int64_t ldl, const sgemm_moe_router *router,
                    int32_t *experts, float *weights, hipStream_t stream);

/* dlogits (T x E) for the gradient dweights of the weights, both T x top like
 * experts and weights, which are what sgemm_moe_route gave for these logits and
 * this router (scoring, renormalize and scale are read).  weights is read with
 * renormalize only, and logits are not read with renormalize and a softmax; they
 * may be NULL otherwise.  A choice outside 0 .. E-1 has no gradient; the terms of
 * an expert chosen twice add up.  The bias has no gradient.  dlogits may be logits
 * itself (same pointer, same leading dimension), or must not overlap it. */
int sgemm_moe_route_backward(int64_t T, int64_t E, int64_t top,
                             const float *logits, int64_t ldl,
                             const sgemm_moe_router *router,
                             const int32_t *experts, const float *weights,
                             const float *dweights, float *dlogits,
                             int64_t lddl, hipStream_t stream);

/* Sorts n = T·top choices by expert, keeping the order of equal ones.
 *   experts   n expert ids, id_bytes 4 (int32) or 8 (int64) bytes each.
 *   offsets   out, E + 1: expert e's rows are offsets[e] .. offsets[e+1]-1;
 *             offsets[0] = 0.
 *   order     out, n: row -> choice; -1 from row offsets[E] on.
 *   place     out, n: choice -> row; -1 where the choice was dropped.
 *   workspace sgemm_moe_sort_workspace_bytes(n, E) bytes, 4-byte aligned;
 *             less is SGEMM_ERR_INVALID_ARG.
 * n == 0 sets offsets to 0.  E over SGEMM_MOE_MAX_EXPERTS or n of 2^31 - 1024
 * or more is SGEMM_ERR_UNSUPPORTED. */
int sgemm_moe_sort(int64_t n, int64_t E, const void *experts, int id_bytes,
                   int32_t *offsets, int32_t *order, int32_t *place,
                   hipStream_t stream, void *workspace, int64_t workspace_bytes);
int64_t sgemm_moe_sort_workspace_bytes(int64_t n, int64_t E);

/* Xp[place[t*top + j]] = X[t] for each kept choice: X is T x H, Xp T·top x H
 * (its other rows are left as they are). */
int sgemm_moe_permute(int64_t T, int64_t top, int64_t H, const float *X,
                      int64_t ldx, const int32_t *place, float *Xp,
                      int64_t ldxp, hipStream_t stream);

/* Y[t] = sum over j of weights[t*top + j] * Yp[place[t*top + j]], in the order
 * j = 0 .. top-1, over the kept choices (0 when a token has none).  weights
 * NULL: all 1. */
int sgemm_moe_unpermute(int64_t T, int64_t top, int64_t H, const float *Yp,
                        int64_t ldyp, const int32_t *place,
                        const float *weights, float *Y, int64_t ldy,
                        hipStream_t stream);

/* The gradients of sgemm_moe_unpermute: for each kept choice c = t*top + j
 *      dYp[place[c]] = weights[c] * dY[t]
 *      dweights[c]   = sum over h of dY[t][h] * Yp[place[c]][h]
 * and dweights[c] = 0 for a dropped one.  weights NULL: all 1.  dYp or
 * dweights may be NULL (Yp is read only for dweights); dYp may be Yp itself
 * (same pointer, same leading dimension). */
int sgemm_moe_unpermute_backward(int64_t T, int64_t top, int64_t H,
                                 const float *dY, int64_t lddy,
                                 const float *Yp, int64_t ldyp,
                                 const int32_t *place, const float *weights,
                                 float *dYp, int64_t lddyp, float *dweights,
                                 hipStream_t stream);

/* For each group g and each row i in offsets[g] .. offsets[g+1]-1:
 *      Z[i] = A[i]·op(B_g) + bias_g,   C[i] = act(Z[i]) + residual[i]
 *   M         rows of A, C, residual and preact (at least offsets[groups]).
 *   groups    0 .. SGEMM_MOE_MAX_EXPERTS.
 *   offsets   groups + 1, not decreasing.
 *   B         group g's matrix at B + g*stride_b, K x N (N x K with trans_b)
 *             with leading dimension ldb; stride_b at least one matrix's
 *             span.
 * Other arguments as for sgemm_linear; the workspace, as there, is room for K
 * to be split, up to sgemm_grouped_workspace_bytes. */
int sgemm_grouped(int trans_b, int64_t M, int64_t N, int64_t K, int64_t groups,
                  const int32_t *offsets, const float *A, int64_t lda,
                  const float *B, int64_t ldb, int64_t stride_b, float *C,
                  int64_t ldc, const sgemm_epilogue *epilogue,
                  hipStream_t stream, void *workspace, int64_t workspace_bytes);
int64_t sgemm_grouped_workspace_bytes(int trans_b, int64_t M, int64_t N,
                                      int64_t K, int64_t groups);

/* For each group g, with its rows as above: dB_g = A[rows]^T·dZ[rows], K x N
 * (or its transpose, N x K, with trans_b), 0 for a group without rows.
 *   dB        group g's at dB + g*stride_db, leading dimension lddb.
 *   workspace room for the sum over rows to be split, up to
 *             sgemm_grouped_wgrad_workspace_bytes. */
int sgemm_grouped_wgrad(int trans_b, int64_t M, int64_t N, int64_t K,
                        int64_t groups, const int32_t *offsets, const float *A,
                        int64_t lda, const float *dZ, int64_t lddz, float *dB,
                        int64_t lddb, int64_t stride_db, hipStream_t stream,
                        void *workspace, int64_t workspace_bytes);
int64_t sgemm_grouped_wgrad_workspace_bytes(int trans_b, int64_t M, int64_t N,
                                            int64_t K, int64_t groups);

/* sgemm_act_backward over the rows of every group: dZ[i] = dC[i] *
 * act'(preact[i]), and dbias (group g's at dbias + g*lddbias) the sums over
 * each group's rows, 0 for a group without rows. */
int sgemm_grouped_act_backward(int64_t M, int64_t N, int64_t groups,
                               const int32_t *offsets, const float *dC,
                               int64_t lddc, const float *preact, int64_t ldp,
                               int act, float *dZ, int64_t lddz, float *dbias,
                               int64_t lddbias, hipStream_t stream,
                               void *workspace, int64_t workspace_bytes);
int64_t sgemm_grouped_act_backward_workspace_bytes(int64_t M, int64_t N,
                                                   int64_t groups);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_MOE_H */
