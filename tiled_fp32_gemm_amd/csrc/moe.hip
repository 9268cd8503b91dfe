// moe.hip -- the C ABI of include/sgemm_moe.h's routing: argument checks and
// launches.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/sgemm_moe.h"
#include "host.hpp"
#include "kernel_moe.hpp"

namespace {

using namespace sg::host;
using sg::MoveArgs;
using sg::SortArgs;

// One workgroup sorts up to kSortOne choices; more are cut into chunks of
// kSortChunk, or longer ones so that there are at most kSortChunks.
constexpr int64_t kSortOne = 8192;
constexpr int64_t kSortChunk = 1024;
constexpr int64_t kSortChunks = 512;

int64_t sort_chunk(int64_t n) {
  if (n <= kSortOne) return n;
  const int64_t c = cdiv(cdiv(n, kSortChunks), 256) * 256;
  return c > kSortChunk ? c : kSortChunk;
}

int launch(const void* fn, int64_t wgs, int threads, void* args, hipStream_t stream) {
  void* kargs[] = {args};
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(threads), kargs, 0, stream) == hipSuccess
             ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

bool bad(const void* p, int64_t bytes) {
  return bytes > 0 && (p == nullptr || ((uintptr_t)p & 3u));
}

// Sizes of a move, and the spans of a T x H and of a T·top x H matrix.
int check_move(int64_t T, int64_t top, int64_t H, int64_t ld_t, int64_t ld_rows, int64_t& t_bytes,
               int64_t& r_bytes) {
  if (T < 0 || top < 0 || H < 0 || ld_t < (H > 1 ? H : 1) || ld_rows < (H > 1 ? H : 1))
    return SGEMM_ERR_INVALID_ARG;
  if (T > kMaxDim || top > kMaxDim || H > kMaxDim || T * top > kMaxDim)
    return SGEMM_ERR_UNSUPPORTED;
  t_bytes = span_bytes(T, H, ld_t);
  r_bytes = span_bytes(T * top, H, ld_rows);
  return t_bytes < 0 || r_bytes < 0 ? SGEMM_ERR_UNSUPPORTED : SGEMM_OK;
}

int launch_move(const void* fn, MoveArgs& a, hipStream_t stream) {
  const int64_t blocks = cdiv(a.T * cdiv(a.H, 4), 256);
  if (!grid_fits(blocks, 256)) return SGEMM_ERR_UNSUPPORTED;
  return launch(fn, blocks, 256, &a, stream);
}

}  // namespace

extern "C" {

int sgemm_moe_sort(int64_t n, int64_t E, const void* experts, int id_bytes, int32_t* offsets,
                   int32_t* order, int32_t* place, hipStream_t stream, void* workspace,
                   int64_t workspace_bytes) {
  if (n < 0 || E < 1 || (id_bytes != 4 && id_bytes != 8) || workspace_bytes < 0)
    return SGEMM_ERR_INVALID_ARG;
  if (bad(experts, n) || bad(offsets, E) || bad(order, n) || bad(place, n) ||
      ((uintptr_t)experts & (uintptr_t)(id_bytes - 1)))
    return SGEMM_ERR_INVALID_ARG;
  if (E > SGEMM_MOE_MAX_EXPERTS || n > kMaxDim) return SGEMM_ERR_UNSUPPORTED;
  const int64_t need = sgemm_moe_sort_workspace_bytes(n, E);
  if (workspace_bytes < need || bad(workspace, need)) return SGEMM_ERR_INVALID_ARG;
  struct { const void* p; int64_t bytes; } out[4] = {
      {offsets, 4 * (E + 1)}, {order, 4 * n}, {place, 4 * n}, {workspace, need}};
  for (int i = 0; i < 4; ++i) {
    if (overlaps(out[i].p, out[i].bytes, experts, n * id_bytes)) return SGEMM_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return SGEMM_ERR_INVALID_ARG;
  }
  SortArgs a;
  a.experts = experts;
  a.offsets = offsets;
  a.order = order;
  a.place = place;
  a.counts = static_cast<int32_t*>(workspace);
  a.n = (int)n;
  a.E = (int)E;
  a.chunk = (int)sort_chunk(n);
  a.chunks = n == 0 ? 1 : (int)cdiv(n, a.chunk);
  a.bits = 0;
  while ((int64_t(1) << a.bits) < E) ++a.bits;
  const bool wide = id_bytes == 8;
  if (a.chunks == 1)
    return launch(wide ? reinterpret_cast<const void*>(sg::moe_sort_kernel<int64_t, 16>)
                       : reinterpret_cast<const void*>(sg::moe_sort_kernel<int32_t, 16>),
                  1, 1024, &a, stream);
  const int st = launch(wide ? reinterpret_cast<const void*>(sg::moe_count_kernel<int64_t>)
                             : reinterpret_cast<const void*>(sg::moe_count_kernel<int32_t>),
                        a.chunks, 256, &a, stream);
  if (st != SGEMM_OK) return st;
  return launch(wide ? reinterpret_cast<const void*>(sg::moe_sort_kernel<int64_t, 4>)
                     : reinterpret_cast<const void*>(sg::moe_sort_kernel<int32_t, 4>),
                a.chunks, 256, &a, stream);
}

int64_t sgemm_moe_sort_workspace_bytes(int64_t n, int64_t E) {
  if (n <= kSortOne || n > kMaxDim || E < 1 || E > SGEMM_MOE_MAX_EXPERTS) return 0;
  return cdiv(n, sort_chunk(n)) * E * 4;
}

int sgemm_moe_permute(int64_t T, int64_t top, int64_t H, const float* X, int64_t ldx,
                      const int32_t* place, float* Xp, int64_t ldxp, hipStream_t stream) {
  int64_t tb, rb;
  const int st = check_move(T, top, H, ldx, ldxp, tb, rb);
  if (st != SGEMM_OK) return st;
  const int64_t n = T * top;
  if (n == 0 || H == 0) return SGEMM_OK;
  if (bad(X, tb) || bad(place, n) || bad(Xp, rb) || overlaps(X, tb, Xp, rb) ||
      overlaps(place, 4 * n, Xp, rb))
    return SGEMM_ERR_INVALID_ARG;
  MoveArgs a = {};
  a.in = X;
  a.out = Xp;
  a.place = place;
  a.ld_in = ldx;
  a.ld_out = ldxp;
  a.T = T;
  a.top = (int)top;
  a.H = (int)H;
  a.rows = (int)n;
  return launch_move(reinterpret_cast<const void*>(sg::moe_permute_kernel), a, stream);
}

int sgemm_moe_unpermute(int64_t T, int64_t top, int64_t H, const float* Yp, int64_t ldyp,
                        const int32_t* place, const float* weights, float* Y, int64_t ldy,
                        hipStream_t stream) {
  int64_t tb, rb;
  const int st = check_move(T, top, H, ldy, ldyp, tb, rb);
  if (st != SGEMM_OK) return st;
  const int64_t n = T * top, wb = weights ? 4 * n : 0;
  if (T == 0 || H == 0) return SGEMM_OK;
  if (bad(Y, tb) || bad(place, n) || bad(Yp, rb) || bad(weights, wb) || overlaps(Y, tb, Yp, rb) ||
      overlaps(Y, tb, place, 4 * n) || overlaps(Y, tb, weights, wb))
    return SGEMM_ERR_INVALID_ARG;
  MoveArgs a = {};
  a.in = Yp;
  a.out = Y;
  a.place = place;
  a.weights = weights;
  a.ld_in = ldyp;
  a.ld_out = ldy;
  a.T = T;
  a.top = (int)top;
  a.H = (int)H;
  a.rows = (int)n;
  return launch_move(reinterpret_cast<const void*>(sg::moe_unpermute_kernel), a, stream);
}

int sgemm_moe_unpermute_backward(int64_t T, int64_t top, int64_t H, const float* dY, int64_t lddy,
                                 const float* Yp, int64_t ldyp, const int32_t* place,
                                 const float* weights, float* dYp, int64_t lddyp, float* dweights,
                                 hipStream_t stream) {
  int64_t tb, yb = 0, db = 0;
  int st = check_move(T, top, H, lddy, dweights ? ldyp : (H > 1 ? H : 1), tb, yb);
  if (st == SGEMM_OK) st = check_move(T, top, H, lddy, dYp ? lddyp : (H > 1 ? H : 1), tb, db);
  if (st != SGEMM_OK) return st;
  const int64_t n = T * top, wb = weights ? 4 * n : 0, gb = dweights ? 4 * n : 0;
  if (!dweights) yb = 0;
  if (!dYp) db = 0;
  if (n == 0 || (!dYp && !dweights) || (H == 0 && !dweights)) return SGEMM_OK;
  if (bad(dY, tb) || bad(Yp, yb) || bad(place, n) || bad(weights, wb) || bad(dYp, db) ||
      bad(dweights, gb))
    return SGEMM_ERR_INVALID_ARG;
  const bool in_place = dYp == Yp && lddyp == ldyp;
  if (overlaps(dYp, db, dY, tb) || (!in_place && overlaps(dYp, db, Yp, yb)) ||
      overlaps(dYp, db, place, 4 * n) || overlaps(dYp, db, weights, wb) ||
      overlaps(dweights, gb, dY, tb) || overlaps(dweights, gb, Yp, yb) ||
      overlaps(dweights, gb, place, 4 * n) || overlaps(dweights, gb, weights, wb) ||
      overlaps(dweights, gb, dYp, db))
    return SGEMM_ERR_INVALID_ARG;
  MoveArgs a = {};
  a.in = Yp;
  a.grad = dY;
  a.out = dYp;
  a.dweights = dweights;
  a.weights = weights;
  a.place = place;
  a.ld_in = ldyp;
  a.ld_grad = lddy;
  a.ld_out = lddyp;
  a.T = T;
  a.top = (int)top;
  a.H = (int)H;
  a.rows = (int)n;
  const bool narrow = H <= 128;
  const int64_t wgs = cdiv(n, narrow ? 16 : 4);
  if (!grid_fits(wgs, 256)) return SGEMM_ERR_UNSUPPORTED;
  return launch(narrow ? reinterpret_cast<const void*>(sg::moe_unpermute_backward_kernel<16>)
                       : reinterpret_cast<const void*>(sg::moe_unpermute_backward_kernel<64>),
                wgs, 256, &a, stream);
}

}  // extern "C"
