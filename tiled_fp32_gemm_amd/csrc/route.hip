// route.hip -- the C ABI of include/sgemm_moe.h's router: argument checks, kernel
// choice and launch.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "../../include/sgemm_moe.h"
#include "host.hpp"
#include "kernel_route.hpp"

namespace {

using namespace sg::host;
using sg::RouteArgs;

typedef void (*RouteFn)(RouteArgs);

// The lanes of a token and its kernels: for lists of 2, 4 .. 32 choices (no more
// than there are experts), and the gradient.
struct Variant {
  int experts, lanes;   // the most experts
  RouteFn route[5];
  RouteFn backward;
};

template <int G, int V>
constexpr Variant variant() {
  return {4 * G * V, G,
          {sg::route_kernel<G, V, 2>, sg::route_kernel<G, V, 4>, sg::route_kernel<G, V, 8>,
           sg::route_kernel<G, V, 16>, sg::route_kernel<G, V, 4 * G * V < 32 ? 16 : 32>},
          sg::route_backward_kernel<G, V>};
}

const Variant kVariants[] = {variant<4, 1>(), variant<8, 1>(), variant<8, 2>(), variant<8, 4>(),
                             variant<8, 8>(), variant<16, 8>(), variant<32, 8>()};

const Variant& variant_for(int64_t E) {
  int i = 0;
  while (kVariants[i].experts < E) ++i;
  return kVariants[i];
}

bool bad(const void* p, int64_t bytes) {
  return bytes > 0 && (p == nullptr || ((uintptr_t)p & 3u));
}

// What both calls check; `ld` is of a T x E matrix.
int check(int64_t T, int64_t E, int64_t top, int64_t ld, const sgemm_moe_router* r) {
  if (T < 0 || E < 1 || top < 1 || top > E || ld < E || r == nullptr) return SGEMM_ERR_INVALID_ARG;
  if ((r->scoring != SGEMM_SCORE_SOFTMAX && r->scoring != SGEMM_SCORE_SIGMOID) ||
      (r->renormalize & ~1) || !isfinite(r->scale) || r->scale == 0.0f)
    return SGEMM_ERR_INVALID_ARG;
  if (T > kMaxDim || E > SGEMM_MOE_MAX_EXPERTS || top > SGEMM_MOE_MAX_TOP)
    return SGEMM_ERR_UNSUPPORTED;
  return SGEMM_OK;
}

RouteArgs args_of(int64_t T, int64_t E, int64_t top, const float* logits, int64_t ld,
                  const sgemm_moe_router* r) {
  RouteArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.T = T;
  a.E = (int)E;
  a.top = (int)top;
  a.scoring = r->scoring;
  a.renormalize = r->renormalize;
  a.scale = r->scale;
  return a;
}

int launch(RouteFn fn, int64_t T, int lanes, RouteArgs& a, hipStream_t stream) {
  const int64_t wgs = cdiv(T, 256 / lanes);
  if (!grid_fits(wgs, 256)) return SGEMM_ERR_UNSUPPORTED;
  void* kargs[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)wgs), dim3(256), kargs,
                         0, stream) == hipSuccess
             ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int sgemm_moe_route(int64_t T, int64_t E, int64_t top, const float* logits, int64_t ldl,
                    const sgemm_moe_router* router, int32_t* experts, float* weights,
                    hipStream_t stream) {
  const int st = check(T, E, top, ldl, router);
  if (st == SGEMM_ERR_INVALID_ARG) return st;
  const sgemm_moe_router& r = *router;
  if (r.groups < 1 || E % r.groups != 0 || r.top_groups < 1 || r.top_groups > r.groups ||
      r.group_best < 1 || r.group_best > 2 || r.group_best > E / r.groups ||
      top > E / r.groups * r.top_groups)
    return SGEMM_ERR_INVALID_ARG;
  if (st != SGEMM_OK || r.groups > SGEMM_MOE_MAX_GROUPS)
    return st != SGEMM_OK ? st : SGEMM_ERR_UNSUPPORTED;
  if (T == 0) return SGEMM_OK;
  const int64_t lb = span_bytes(T, E, ldl), nb = 4 * T * top, bb = r.bias ? 4 * E : 0;
  if (bad(logits, lb < 0 ? 1 : lb) || bad(experts, nb) || bad(weights, nb) || bad(r.bias, bb))
    return SGEMM_ERR_INVALID_ARG;
  if (lb < 0) return SGEMM_ERR_UNSUPPORTED;
  if (overlaps(experts, nb, logits, lb) || overlaps(weights, nb, logits, lb) ||
      overlaps(experts, nb, r.bias, bb) || overlaps(weights, nb, r.bias, bb) ||
      overlaps(experts, nb, weights, nb))
    return SGEMM_ERR_INVALID_ARG;
  RouteArgs a = args_of(T, E, top, logits, ldl, router);
  a.bias = r.bias;
  a.experts = experts;
  a.weights = weights;
  a.groups = r.groups;
  a.top_groups = r.top_groups;
  a.group_best = r.group_best;
  a.size = (int)(E / r.groups);
  a.per = (int)cdiv(1 << 20, a.size);
  const Variant& v = variant_for(E);
  int list = 0;   // 2^(list + 1) choices
  while ((2 << list) < top) ++list;
  return launch(v.route[list], T, v.lanes, a, stream);
}

int sgemm_moe_route_backward(int64_t T, int64_t E, int64_t top, const float* logits, int64_t ldl,
                             const sgemm_moe_router* router, const int32_t* experts,
                             const float* weights, const float* dweights, float* dlogits,
                             int64_t lddl, hipStream_t stream) {
  const bool unread = router && router->renormalize && router->scoring == SGEMM_SCORE_SOFTMAX;
  const int st = check(T, E, top, unread ? E : ldl, router);
  if (st == SGEMM_ERR_INVALID_ARG || lddl < E) return SGEMM_ERR_INVALID_ARG;
  if (st != SGEMM_OK) return st;
  if (T == 0) return SGEMM_OK;
  const int64_t lb = unread ? 0 : span_bytes(T, E, ldl), db = span_bytes(T, E, lddl);
  const int64_t nb = 4 * T * top, wb = router->renormalize ? nb : 0;
  if (bad(logits, lb < 0 ? 1 : lb) || bad(dlogits, db < 0 ? 1 : db) || bad(experts, nb) ||
      bad(dweights, nb) || bad(weights, wb))
    return SGEMM_ERR_INVALID_ARG;
  if (lb < 0 || db < 0) return SGEMM_ERR_UNSUPPORTED;
  const bool in_place = dlogits == logits && (T == 1 || lddl == ldl);
  if ((!in_place && overlaps(dlogits, db, logits, lb)) || overlaps(dlogits, db, experts, nb) ||
      overlaps(dlogits, db, dweights, nb) || overlaps(dlogits, db, weights, wb))
    return SGEMM_ERR_INVALID_ARG;
  RouteArgs a = args_of(T, E, top, logits, ldl, router);
  a.experts = const_cast<int32_t*>(experts);
  a.weights = const_cast<float*>(weights);
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.ldd = lddl;
  const Variant& v = variant_for(E);
  return launch(v.backward, T, v.lanes, a, stream);
}

}  // extern "C"
