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

#include "activation.hpp"
#include "rows.hpp"
#include "xent_args.hpp"

namespace sg {

// A workgroup takes a chunk of tokens, kXentBlock at a time: counts the rows with a
// target before its chunk, numbers its own, and its waves copy their rows of X.
constexpr int kXentBlock = 32;

__global__ void __launch_bounds__(256) xent_gather_kernel(XentGatherArgs a) {
  __shared__ int part[4];
  __shared__ int row_of[kXentBlock];
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
    const int64_t t = t0 + lane;
    const int target = lane < kXentBlock && t < last ? a.targets.of(t) : -1;
    const uint64_t kept = __ballot(target >= 0);   // the same in every wave
    const int row = target >= 0 ? before + __popcll(kept & ((uint64_t(1) << lane) - 1)) : -1;
    if (wave == 0 && lane < kXentBlock && t < last) {
      row_of[lane] = row;
      a.rows.place[t] = row;
      if (row >= 0) {
        a.rows.order[row] = (int)t;
        a.rows.target[row] = target;
        if (a.lse) {
          a.rows.lse[row] = a.lse[t];
          a.rows.grad[row] = a.dloss[t];
        }
      }
    }
    __syncthreads();
    for (int i = wave; i < kXentBlock && t0 + i < last; i += 4) {
      const int to = row_of[i];
      if (to < 0) continue;
      const float* const x = a.X + (t0 + i) * a.ldx;
      float* const y = a.rows.X + (int64_t)to * a.H;
#pragma unroll 4
      for (int64_t col = 4 * lane; col < a.H; col += 256)
        store_upto(y + col, (int)min((int64_t)4, a.H - col),
                   load_upto_once(x + col, (int)min((int64_t)4, a.H - col)));
    }
    before += __popcll(kept);
    __syncthreads();   // row_of is read before it is written again
  }
  if (tid == 0 && last == a.T) {
    a.rows.offsets[0] = 0;
    a.rows.offsets[1] = before;
  }
}

// The strips of kXentLossRows tokens' rows: part p of a token takes strips p,
// p + kXentLossParts .., eight at a time, and the parts meet by halves.
constexpr int kXentLossRows = 16, kXentLossParts = 64;

__global__ void __launch_bounds__(kXentLossRows * kXentLossParts)
xent_loss_kernel(XentLossArgs a) {
  constexpr int U = 8;
  __shared__ float all_m[kXentLossParts][kXentLossRows], all_s[kXentLossParts][kXentLossRows];
  const int i = (int)threadIdx.x % kXentLossRows, p = (int)threadIdx.x / kXentLossRows;
  const int64_t t = (int64_t)blockIdx.x * kXentLossRows + i;
  const bool kept = t < a.T && a.targets.of(t) >= 0;
  const int64_t row = !kept ? 0 : a.place ? a.place[t] : t;
  float m = -FLT_MAX, s = 0.0f;
  auto join = [&](float m2, float s2) {
    const float top = fmaxf(m, m2);
    s = s * exp_accurate(m - top) + s2 * exp_accurate(m2 - top);
    m = top;
  };
  if (kept) {
    for (int j0 = p; j0 < a.strips; j0 += U * kXentLossParts) {
      float mm[U], ss[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * kXentLossParts;
        mm[u] = -FLT_MAX;
        ss[u] = 0.0f;
        if (j < a.strips) {
          mm[u] = a.max[(int64_t)j * a.ld_strip + row];
          ss[u] = a.sum[(int64_t)j * a.ld_strip + row];
        }
      }
      float top = m;
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, mm[u]);
      s *= exp_accurate(m - top);
#pragma unroll
      for (int u = 0; u < U; ++u) s += ss[u] * exp_accurate(mm[u] - top);
      m = top;
    }
  }
  all_m[p][i] = m;
  all_s[p][i] = s;
  for (int half = kXentLossParts / 2; half > 0; half /= 2) {
    __syncthreads();
    if (p < half) {
      join(all_m[p + half][i], all_s[p + half][i]);
      all_m[p][i] = m;
      all_s[p][i] = s;
    }
  }
  if (p > 0 || t >= a.T) return;
  const float rest = logf(s);
  // Before m and log s are rounded together.
  a.loss[t] = kept ? (m - a.hit[row]) + rest : 0.0f;
  if (a.lse) a.lse[t] = kept ? m + rest : 0.0f;
}

}  // namespace sg
