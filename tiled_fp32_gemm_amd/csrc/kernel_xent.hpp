// kernel_xent.hpp -- softmax cross entropy over a product's columns, without the
// product in memory.
//
// With z = X·op(B) (T x V), lse = log sum exp z and the target's logit z_t of a
// row:  loss = lse - z_t,  dz = (exp(z - lse) - [column is the target]) dloss.
//
// Forward, product_kernel ends in XentStats: each wave has 32 or 64 columns of its
// rows (a strip) and leaves, for each row, their largest logit m and the sum of
// exp(z - m); the lane that has the target's column leaves it.  xent_loss_kernel
// joins a row's strips: (m, s) and (m', s') make (M, s e^(m - M) + s' e^(m' - M)).
// Backward, the product is made again, a piece of the vocabulary at a time, and
// ends in XentGrad, which stores the piece's dz; two products of the library take
// it on to dX and dB.
//
// Rows without a target are left out of the products altogether: xent_gather_kernel
// copies the others' rows of X together, and how many there are stays on the
// device.  A padded or masked row costs nothing and, whatever it holds, reaches no
// gradient.
#pragma once

#include <float.h>

#include "rows.hpp"
#include "xent_args.hpp"

namespace sg {

// A workgroup takes a chunk of tokens, kXentBlock at a time: counts the rows with a
// target before its chunk, numbers its own, and its waves copy their rows of X, two
// each.
constexpr int kXentBlock = 8;

__global__ void __launch_bounds__(256) xent_gather_kernel(XentGatherArgs a) {
  __shared__ int part[4];
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t first = (int64_t)blockIdx.x * a.chunk, last = min(first + a.chunk, a.T);
  int before = 0;
#pragma unroll 8
  for (int64_t t = tid; t < first; t += 256) before += a.targets.of(t) >= 0 ? 1 : 0;
  for (int d = 32; d > 0; d >>= 1) before += __shfl_xor(before, d);
  if (lane == 0) part[wave] = before;
  __syncthreads();
  before = part[0] + part[1] + part[2] + part[3];
  for (int64_t t0 = first; t0 < last; t0 += kXentBlock) {
    // Every wave numbers the block's rows for itself.
    const int64_t t = t0 + lane;
    const int target = lane < kXentBlock && t < last ? a.targets.of(t) : -1;
    const uint64_t kept = __ballot(target >= 0);
    const int row = target >= 0 ? before + __popcll(kept & ((uint64_t(1) << lane) - 1)) : -1;
    if (wave == 0 && lane < kXentBlock && t < last) {
      a.rows.place[t] = row;
      if (row >= 0) {
        if (a.lse) {
          const float ref = a.lse[t] * kLog2e;
          a.rows.row[row] = {target, ref, fmaf(a.lse[t], kLog2e, -ref), a.dloss[t]};
        } else {
          a.rows.target[row] = target;
        }
      }
    }
    const int to0 = __shfl(row, 2 * wave), to1 = __shfl(row, 2 * wave + 1);
    const float* const x = a.X + (t0 + 2 * wave) * a.ldx;
    constexpr int U = 4;   // groups of each row in flight
    for (int64_t c0 = 4 * lane; c0 < a.H; c0 += U * 256) {
      f32x4 v[2][U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t col = c0 + u * 256;
        const int n = (int)min((int64_t)4, a.H - col);
        if (n > 0 && to0 >= 0) v[0][u] = load_upto_once(x + col, n);
        if (n > 0 && to1 >= 0) v[1][u] = load_upto_once(x + a.ldx + col, n);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t col = c0 + u * 256;
        const int n = (int)min((int64_t)4, a.H - col);
        if (n > 0 && to0 >= 0) store_upto(a.rows.X + (int64_t)to0 * a.H + col, n, v[0][u]);
        if (n > 0 && to1 >= 0) store_upto(a.rows.X + (int64_t)to1 * a.H + col, n, v[1][u]);
      }
    }
    before += __popcll(kept);
  }
  if (tid == 0 && last == a.T) {
    a.rows.offsets[0] = 0;
    a.rows.offsets[1] = before;
  }
}

// The strips of kXentLossRows tokens' rows: part p of a token takes strips p,
// p + kXentLossParts .., sixteen at a time, and the parts meet by halves.
constexpr int kXentLossRows = 16, kXentLossParts = 64;

__global__ void __launch_bounds__(kXentLossRows * kXentLossParts)
xent_loss_kernel(XentLossArgs a) {
  constexpr int U = 16;
  __shared__ float all_m[kXentLossParts][kXentLossRows], all_s[kXentLossParts][kXentLossRows];
  const int i = (int)threadIdx.x % kXentLossRows, p = (int)threadIdx.x / kXentLossRows;
  const int64_t t = (int64_t)blockIdx.x * kXentLossRows + i;
  const bool kept = t < a.T && a.targets.of(t) >= 0;
  const int64_t row = !kept ? 0 : a.place ? a.place[t] : t;
  const float hit = kept && p == 0 ? a.hit[row] : 0.0f;
  float m = -INFINITY, s = 0.0f;   // the sum relative to m's reference
  if (kept) {
    for (int j0 = p; j0 < a.strips; j0 += U * kXentLossParts) {
      float mm[U], ss[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * kXentLossParts;
        mm[u] = -INFINITY;
        ss[u] = 0.0f;
        if (j < a.strips) {
          mm[u] = a.max[(int64_t)j * a.ld_strip + row];
          ss[u] = a.sum[(int64_t)j * a.ld_strip + row];
        }
      }
      float top = m;
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, mm[u]);
      const float ref = xent_reference(top);
      s *= __builtin_amdgcn_exp2f(xent_reference(m) - ref);
#pragma unroll
      for (int u = 0; u < U; ++u)
        s += ss[u] * __builtin_amdgcn_exp2f(xent_reference(mm[u]) - ref);
      m = top;
    }
  }
  all_m[p][i] = m;
  all_s[p][i] = s;
  for (int half = kXentLossParts / 2; half > 0; half /= 2) {
    __syncthreads();
    if (p < half) {
      const float m2 = all_m[p + half][i], s2 = all_s[p + half][i], top = fmaxf(m, m2);
      const float ref = xent_reference(top);
      s = s * __builtin_amdgcn_exp2f(xent_reference(m) - ref) +
          s2 * __builtin_amdgcn_exp2f(xent_reference(m2) - ref);
      m = top;
      all_m[p][i] = m;
      all_s[p][i] = s;
    }
  }
  if (p > 0 || t >= a.T) return;
  // log s, and what the rounding of m's reference moved s by.
  m = fminf(fmaxf(m, -FLT_MAX), FLT_MAX);
  const float rest = (log2f(s) - fmaf(m, kLog2e, -xent_reference(m))) * 0.693147182f;
  // Before m and the rest are rounded together.
  a.loss[t] = kept ? (m - hit) + rest : 0.0f;
  if (a.lse) a.lse[t] = kept ? m + rest : 0.0f;
}

}  // namespace sg
