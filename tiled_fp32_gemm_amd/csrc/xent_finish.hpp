// xent_finish.hpp -- the cross entropy's epilogues of product_kernel (see
// kernel_xent.hpp): what a wave does with four columns of a row of logits.
#pragma once

#include "lanes.hpp"
#include "rows.hpp"
#include "xent_args.hpp"

namespace sg {

// f over the 8 or 16 lanes that share a row, for every row, all lanes active.
template <int CTRL, int IT, class F>
__device__ __forceinline__ void strip_step(float (&v)[IT], F f) {
#pragma unroll
  for (int it = 0; it < IT; ++it) v[it] = f(v[it], dpp_of<CTRL>(v[it]));
}
template <int LPR, int IT, class F>
__device__ __forceinline__ void strip_each(float (&v)[IT], F f) {
  static_assert(LPR == 8 || LPR == 16, "lanes of a row");
  strip_step<0xB1, IT>(v, f);    // quad_perm 1, 0, 3, 2
  strip_step<0x4E, IT>(v, f);    // quad_perm 2, 3, 0, 1
  strip_step<0x141, IT>(v, f);   // row_half_mirror
  if constexpr (LPR == 16) strip_step<0x140, IT>(v, f);   // row_mirror
}

// Exponentials here are powers of two of fma(z, kLog2e, -ref): two instructions, with
// an error of half a step of the exponent and 0.22 of one of z - its reference (what
// kLog2e is off).  A row's reference is its largest logit times kLog2e, rounded; what
// that rounding leaves is put right once a row (xent_loss_kernel).

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
        target[it] = g.target ? g.target[row] : g.targets.of(row);
      }
    }
  }
  // All rows' steps side by side, so that they wait for each other's DPP results.
  template <int LPR, int IT>
  __device__ __forceinline__ void rows(const Args& g, f32x4 (&v)[IT], const int (&at)[IT],
                                       int row0, int m_left, int col, int cols, int l) const {
    float m[IT], s[IT];
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int mine = target[it] - col;   // a target is one of the columns
      if (mine >= 0 && mine < 4 && at[it] < m_left) {
        const float z = mine < 2 ? (mine == 0 ? v[it][0] : v[it][1])
                                 : (mine == 2 ? v[it][2] : v[it][3]);
        g.hit[row0 + at[it]] = z;
      }
    }
#pragma unroll
    for (int it = 0; it < IT; ++it) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[it][e] = e < cols ? v[it][e] : -INFINITY;
      m[it] = fmaxf(fmaxf(v[it][0], v[it][1]), fmaxf(v[it][2], v[it][3]));
    }
    strip_each<LPR, IT>(m, [](float x, float y) { return fmaxf(x, y); });
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const float ref = xent_reference(m[it]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[it][e] = __builtin_amdgcn_exp2f(fmaf(v[it][e], kLog2e, -ref));
      s[it] = (v[it][0] + v[it][1]) + (v[it][2] + v[it][3]);
    }
    strip_each<LPR, IT>(s, [](float x, float y) { return x + y; });
    if (l != 0 || cols <= 0) return;
    const int64_t strip = (int64_t)(col / (4 * LPR)) * g.ld_strip + row0;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if (at[it] < m_left) {
        g.max[strip + at[it]] = m[it];
        g.sum[strip + at[it]] = s[it];
      }
    }
  }
};

struct XentGrad {
  using Args = XentProductArgs;
  XentRow info[8];

  template <int IT>
  __device__ __forceinline__ void load(const Args& g, const int (&at)[IT], int row0, int m_left) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      info[it] = {-1, 0.0f, 0.0f, 0.0f};
      if (at[it] < m_left)
        info[it] = __builtin_bit_cast(
            XentRow, f32x4(*reinterpret_cast<const f32x4u*>(g.row + row0 + at[it])));
    }
  }
  template <int LPR, int IT>
  __device__ __forceinline__ void rows(const Args& g, f32x4 (&v)[IT], const int (&at)[IT],
                                       int row0, int m_left, int col, int cols, int) const {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int mine = info[it].target - g.column0 - col;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = __builtin_amdgcn_exp2f(fmaf(v[it][e], kLog2e, -info[it].ref) -
                                             info[it].rest);
        v[it][e] = (p - (mine == e ? 1.0f : 0.0f)) * info[it].grad;
      }
    }
    if (cols <= 0) return;
    float* const out = g.C + (int64_t)row0 * g.ldc + col;
#pragma unroll
    for (int it = 0; it < IT; ++it)
      if (at[it] < m_left) store_upto(out + (int64_t)at[it] * g.ldc, cols, v[it]);
  }
};

}  // namespace sg
