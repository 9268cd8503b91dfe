// norm.hip -- the C ABI of include/sgemm_norm.h: argument checks, kernel choice
// and launch.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/sgemm_norm.h"
#include "host.hpp"
#include "kernel_norm.hpp"

namespace {

using namespace sg::host;
using sg::NormArgs;
using sg::NormBackwardArgs;

struct Span {
  const void* p;
  int64_t bytes;   // 0: not touched; -1: beyond int64
};

bool overlaps(const Span& a, const Span& b) {
  return sg::host::overlaps(a.p, a.bytes, b.p, b.bytes);
}

// A span that is touched has to be there and aligned; one beyond int64 is
// unsupported.
int check_spans(const Span* s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i].bytes != 0 && (s[i].p == nullptr || ((uintptr_t)s[i].p & 3u)))
      return SGEMM_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (s[i].bytes < 0) return SGEMM_ERR_UNSUPPORTED;
  return SGEMM_OK;
}

// The outputs overlap no input and no other output, but where they may be one
// (same pointer, same leading dimension: `same` marks the input).
bool apart(const Span* in, int ins, const bool* same, const Span* out, int outs) {
  for (int o = 0; o < outs; ++o) {
    for (int i = 0; i < ins; ++i)
      if (!(o == 0 && same[i]) && overlaps(out[o], in[i])) return false;
    for (int p = 0; p < o; ++p)
      if (overlaps(out[o], out[p])) return false;
  }
  return true;
}

template <class Fn>
struct Variant {
  int cols, lanes, threads;   // columns it holds; lanes of a row
  Fn fn;
};

typedef void (*NormFn)(NormArgs);
typedef void (*NormBackwardFn)(NormBackwardArgs);

#define NORM_VARIANT(fn, L, V) {4 * L * V, L, sg::kNormThreads<L>, sg::fn<L, V>}
const Variant<NormFn> kForward[] = {
    NORM_VARIANT(norm_kernel, 16, 1),  NORM_VARIANT(norm_kernel, 16, 2),
    NORM_VARIANT(norm_kernel, 64, 1),  NORM_VARIANT(norm_kernel, 64, 2),
    NORM_VARIANT(norm_kernel, 64, 4),  NORM_VARIANT(norm_kernel, 256, 2),
    NORM_VARIANT(norm_kernel, 256, 4), NORM_VARIANT(norm_kernel, 1024, 2),
    NORM_VARIANT(norm_kernel, 1024, 4)};
const Variant<NormBackwardFn> kBackward[] = {
    NORM_VARIANT(norm_backward_kernel, 16, 1),  NORM_VARIANT(norm_backward_kernel, 16, 2),
    NORM_VARIANT(norm_backward_kernel, 64, 1),  NORM_VARIANT(norm_backward_kernel, 64, 2),
    NORM_VARIANT(norm_backward_kernel, 64, 4),  NORM_VARIANT(norm_backward_kernel, 256, 2),
    NORM_VARIANT(norm_backward_kernel, 256, 4), NORM_VARIANT(norm_backward_kernel, 1024, 2)};
#undef NORM_VARIANT

// The narrowest variant that holds a row; null: none does.
template <class Fn, int n>
const Variant<Fn>* variant_for(const Variant<Fn> (&table)[n], int64_t N) {
  for (const Variant<Fn>& v : table)
    if (N <= v.cols) return &v;
  return nullptr;
}

// Workgroups that take the rows in turn.
int64_t norm_grid(int64_t M, int lanes, int threads) {
  const int64_t all = cdiv(M, threads / lanes), most = kCUs * 8 * 256 / threads;
  return all < most ? all : most;
}

// Rows of sums that the backward pass leaves in its workspace.
int64_t norm_spans(int64_t M, int64_t N) {
  const Variant<NormBackwardFn>* v = variant_for(kBackward, N);
  const int64_t beside = v ? v->threads / v->lanes : 1;
  const int64_t all = cdiv(M, beside), least = cdiv(all, sg::kNormRun);
  // More of them fill the chip better, fewer leave less to write and to add up: by
  // 64 lanes and more than 512 columns, or 256 lanes, two a CU (us, both kernels, with
  // 256, 512 and 1024 of them: 8192 x 1024 26.5 / 23.4 / 27.3, 4096 x 4096 49.9 / 43.2 /
  // 52.2, 1000 x 4096 20.6 / 21.4 / 29.3), of narrower rows four (60000 x 256 69 / 41 / 36,
  // 200000 x 64 57 / 34 / 30), of wider ones one (3000 x 8192 62 / 71 / 87).
  int64_t most = kCUs * (N <= 512 ? 4 : N <= 4096 ? 2 : 1);
  if (!v) most = cdiv(4 * kCUs, cdiv(N, sg::kNormWideCols));
  if (most < least) most = least;
  return all < most ? all : most;
}

bool sizes_ok(int64_t M, int64_t N) { return M >= 0 && N >= 0 && M <= kMaxDim && N <= kMaxDim; }

int launch(const void* fn, int64_t wgs, int threads, void* args, hipStream_t stream) {
  if (!grid_fits(wgs, threads)) return SGEMM_ERR_UNSUPPORTED;
  void* kargs[] = {args};
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(threads), kargs, 0, stream) == hipSuccess
             ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int sgemm_layer_norm(int64_t M, int64_t N, const float* X, int64_t ldx, const float* weight,
                     const float* bias, float eps, float* Y, int64_t ldy, float* mean,
                     float* rstd, hipStream_t stream) {
  const int64_t n1 = N > 1 ? N : 1;
  if (M < 0 || N < 0 || ldx < n1 || ldy < n1 || !(eps >= 0.0f)) return SGEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return SGEMM_OK;
  const Span in[] = {{X, span_bytes(M, N, ldx)},
                     {weight, weight ? span_bytes(1, N, N) : 0},
                     {bias, bias ? span_bytes(1, N, N) : 0}};
  const Span out[] = {{Y, span_bytes(M, N, ldy)},
                      {mean, mean ? span_bytes(1, M, M) : 0},
                      {rstd, rstd ? span_bytes(1, M, M) : 0}};
  int st = check_spans(in, 3);
  if (st == SGEMM_OK) st = check_spans(out, 3);
  if (st != SGEMM_OK) return st;
  if (!sizes_ok(M, N)) return SGEMM_ERR_UNSUPPORTED;
  const bool same[] = {X == Y && (M == 1 || ldx == ldy), false, false};
  if (!apart(in, 3, same, out, 3)) return SGEMM_ERR_INVALID_ARG;
  NormArgs a;
  a.X = X;
  a.weight = weight;
  a.bias = bias;
  a.Y = Y;
  a.mean = mean;
  a.rstd = rstd;
  a.ldx = ldx;
  a.ldy = ldy;
  a.M = M;
  a.N = (int)N;
  a.eps = eps;
  if (const Variant<NormFn>* v = variant_for(kForward, N))
    return launch(reinterpret_cast<const void*>(v->fn), norm_grid(M, v->lanes, v->threads),
                  v->threads, &a, stream);
  return launch(reinterpret_cast<const void*>(sg::norm_wide_kernel), M, 1024, &a, stream);
}

int64_t sgemm_layer_norm_backward_workspace_bytes(int64_t M, int64_t N) {
  if (!sizes_ok(M, N) || M == 0 || N == 0) return 0;
  return norm_spans(M, N) * 2 * N * 4;
}

int sgemm_layer_norm_backward(int64_t M, int64_t N, const float* dY, int64_t lddy, const float* X,
                              int64_t ldx, const float* mean, const float* rstd,
                              const float* weight, const float* residual, int64_t ldr, float* dX,
                              int64_t lddx, float* dweight, float* dbias, hipStream_t stream,
                              void* workspace, int64_t workspace_bytes) {
  const int64_t n1 = N > 1 ? N : 1;
  if (M < 0 || N < 0 || lddy < n1 || ldx < n1 || (residual && ldr < n1) || (dX && lddx < n1) ||
      workspace_bytes < 0)
    return SGEMM_ERR_INVALID_ARG;
  const bool sums = dweight || dbias;
  if (N == 0 || (!dX && !sums) || (M == 0 && !sums)) return SGEMM_OK;
  if (!dX) residual = nullptr;
  const int64_t need = sums ? sgemm_layer_norm_backward_workspace_bytes(M, N) : 0;
  const Span in[] = {{dY, span_bytes(M, N, lddy)},
                     {X, span_bytes(M, N, ldx)},
                     {residual, residual ? span_bytes(M, N, ldr) : 0},
                     {mean, span_bytes(1, M, M)},
                     {rstd, span_bytes(1, M, M)},
                     {weight, weight ? span_bytes(1, N, N) : 0}};
  const Span out[] = {{dX, dX ? span_bytes(M, N, lddx) : 0},
                      {dweight, dweight ? span_bytes(1, N, N) : 0},
                      {dbias, dbias ? span_bytes(1, N, N) : 0},
                      {workspace, need}};
  int st = check_spans(in, 6);
  if (st == SGEMM_OK) st = check_spans(out, 4);
  if (st != SGEMM_OK) return st;
  if (!sizes_ok(M, N)) return SGEMM_ERR_UNSUPPORTED;
  if (workspace_bytes < need) return SGEMM_ERR_INVALID_ARG;
  auto on = [&](const float* p, int64_t ld) { return p == dX && (M == 1 || ld == lddx); };
  const bool same[] = {on(dY, lddy), on(X, ldx), on(residual, ldr), false, false, false};
  if (!apart(in, 6, same, out, 4)) return SGEMM_ERR_INVALID_ARG;
  NormBackwardArgs a;
  a.dY = dY;
  a.X = X;
  a.mean = mean;
  a.rstd = rstd;
  a.weight = weight;
  a.residual = residual;
  a.dX = dX;
  a.W = sums && M > 0 ? static_cast<float*>(workspace) : nullptr;
  a.dweight = dweight;
  a.dbias = dbias;
  a.lddy = lddy;
  a.ldx = ldx;
  a.ldr = ldr;
  a.lddx = lddx;
  a.M = M;
  a.N = (int)N;
  a.spans = M > 0 ? (int)norm_spans(M, N) : 0;
  const int64_t columns = cdiv(2 * N, sg::kNormSumCols);
  const Variant<NormBackwardFn>* v = variant_for(kBackward, N);
  // Checked before the first launch.
  const int64_t wide = (int64_t)a.spans * cdiv(N, sg::kNormWideCols);
  if ((sums && !grid_fits(columns, 1024)) ||
      (v ? !grid_fits(a.spans, v->threads)
         : !grid_fits(wide, 256) || (dX && !grid_fits(M, 1024))))
    return SGEMM_ERR_UNSUPPORTED;
  if (M > 0 && v) {
    st = launch(reinterpret_cast<const void*>(v->fn), a.spans, v->threads, &a, stream);
  } else if (M > 0) {
    // The sums first: dX may lie on what they read.
    if (sums)
      st = launch(reinterpret_cast<const void*>(sg::norm_wide_sums_kernel), wide, 256, &a, stream);
    if (st == SGEMM_OK && dX)
      st = launch(reinterpret_cast<const void*>(sg::norm_wide_backward_kernel), M, 1024, &a,
                  stream);
  }
  if (st != SGEMM_OK || !sums) return st;
  return launch(reinterpret_cast<const void*>(sg::norm_sum_kernel), columns, 1024, &a, stream);
}

}  // extern "C"
