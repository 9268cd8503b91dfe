// xent_finish.hpp -- the cross entropy's epilogues of product_kernel (see
// kernel_xent.hpp): what a wave does with four columns of a row of logits.
#pragma once

#include <float.h>

#include "activation.hpp"
#include "lanes.hpp"
#include "rows.hpp"
#include "xent_args.hpp"

namespace sg {

// Over the 8 or 16 lanes that share a row, all of them active.
template <int LPR>
__device__ __forceinline__ float strip_sum(float v) {
  static_assert(LPR == 8 || LPR == 16, "lanes of a row");
  v += dpp_of<0xB1>(v);
  v += dpp_of<0x4E>(v);
  v += dpp_of<0x141>(v);
  if constexpr (LPR == 16) v += dpp_of<0x140>(v);
  return v;
}
template <int LPR>
__device__ __forceinline__ float strip_max(float v) {
  v = fmaxf(v, dpp_of<0xB1>(v));
  v = fmaxf(v, dpp_of<0x4E>(v));
  v = fmaxf(v, dpp_of<0x141>(v));
  if constexpr (LPR == 16) v = fmaxf(v, dpp_of<0x140>(v));
  return v;
}

// Finite, so that a row of infinities subtracts no infinity from itself.
__device__ __forceinline__ float finite_max(float m) {
  return fminf(fmaxf(m, -FLT_MAX), FLT_MAX);
}

struct XentStats {
  using Args = XentProductArgs;
  int target[8];

  template <int IT>
  __device__ __forceinline__ void load(const Args& g, const int (&at)[IT], int row0, int m_left) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      target[it] = -1;
      if (at[it] < m_left) {
        const int row = row0 + at[it];
        target[it] = g.targets.of(g.order ? g.order[row] : row);
      }
    }
  }
  template <int LPR>
  __device__ __forceinline__ void row(const Args& g, int it, f32x4 v, int row0, int at, int col,
                                      int cols, int l) const {
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < cols) m = fmaxf(m, v[e]);
    m = finite_max(strip_max<LPR>(m));
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) s += e < cols ? exp_accurate(v[e] - m) : 0.0f;
    s = strip_sum<LPR>(s);
    if (at < 0) return;
    const int64_t row = row0 + at;
    if (l == 0 && cols > 0) {
      const int64_t place = (int64_t)(col / (4 * LPR)) * g.ld_strip + row;
      g.max[place] = m;
      g.sum[place] = s;
    }
    const int mine = target[it] - col;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (mine == e && e < cols) g.hit[row] = v[e];
  }
};

struct XentGrad {
  using Args = XentProductArgs;
  int target[8];
  float lse[8], grad[8];

  template <int IT>
  __device__ __forceinline__ void load(const Args& g, const int (&at)[IT], int row0, int m_left) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      target[it] = -1;
      lse[it] = grad[it] = 0.0f;
      if (at[it] < m_left) {
        target[it] = g.target[row0 + at[it]];
        lse[it] = g.lse[row0 + at[it]];
        grad[it] = g.grad[row0 + at[it]];
      }
    }
  }
  template <int LPR>
  __device__ __forceinline__ void row(const Args& g, int it, f32x4 v, int row0, int at, int col,
                                      int cols, int) const {
    if (at < 0 || cols <= 0) return;
    const int mine = target[it] - g.column0 - col;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = (exp_accurate(v[e] - lse[it]) - (mine == e ? 1.0f : 0.0f)) * grad[it];
    store_upto(g.C + (int64_t)(row0 + at) * g.ldc + col, cols, v);
  }
};

}  // namespace sg
