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
// Where tiles of all of K are too few to fill the chip, or a few rows are faster
// without tiles, the product is left in planes, one for each part of a split K, and a
// pass over them (xent_planes_*) adds them up and does the same.
//
// Rows without a target are left out of the products altogether: xent_place_kernel or
// xent_gather_kernel numbers the others, whose rows of X are copied together; how many
// there are stays on the device.  A padded or masked row costs nothing and, whatever it
// holds, reaches no gradient.
//
// Bound by the matrix pipe for many rows, by reading B for a few.  Measured on MI355X
// with B stored V x H, H = 1024, V = 32768 (averages of forty passes over three states in
// turn): 6144 rows forward 2910 us (142 TFLOP/s; 2823 at least, 146), numbering and copying
// them 6 + 12, joining 512 strips of 8192 tokens 12; the gradient of half that vocabulary
// for 8192 rows 1927 us, 95 more than a product, of which dz's 512 MiB are most; 16 rows
// forward 28.8 us (4.7 TB/s) and 4.4 for their 1024 strips; 64 rows 43.8 + 5.4; 1000 rows
// 545 (123 TFLOP/s), 6 for their copies and 6 for the strips.
#pragma once

#include <float.h>

#include "lanes.hpp"
#include "rows.hpp"
#include "xent_args.hpp"

namespace sg {

// Numbers the rows with a target.  A workgroup takes a chunk of tokens, a token a
// thread at a time, after it has counted the rows of all the chunks before its own.
constexpr int kXentPlaceThreads = 256;

__global__ void __launch_bounds__(kXentPlaceThreads) xent_place_kernel(XentPlaceArgs a) {
  constexpr int NT = kXentPlaceThreads, WAVES = NT / 64;
  __shared__ int before[WAVES], own[2][WAVES];
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t first = (int64_t)blockIdx.x * a.chunk, last = min(first + a.chunk, a.T);
  int n = 0;
  auto count = [&](auto* ids) {
#pragma unroll 16
    for (int64_t i = tid; i < first; i += NT) n += ids[i] >= 0 && ids[i] < a.targets.V ? 1 : 0;
  };
  if (a.targets.wide) count(static_cast<const int64_t*>(a.targets.ids));
  else count(static_cast<const int32_t*>(a.targets.ids));
  for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d);
  if (lane == 0) before[wave] = n;
  __syncthreads();
  int next = 0;   // the row after those so far
  for (int w = 0; w < WAVES; ++w) next += before[w];
  int odd = 0;    // a wave may still read the counts of the time before
  for (int64_t t0 = first; t0 < last; t0 += NT, odd ^= 1) {
    const int64_t t = t0 + tid;
    const int target = t < last ? a.targets.of(t) : -1;
    const uint64_t kept = __ballot(target >= 0);
    if (lane == 0) own[odd][wave] = __popcll(kept);
    __syncthreads();
    int row = next + __popcll(kept & ((uint64_t(1) << lane) - 1));
    for (int w = 0; w < WAVES; ++w) {
      if (w < wave) row += own[odd][w];
      next += own[odd][w];
    }
    if (t < last) a.rows.place[t] = target >= 0 ? row : -1;
    if (target < 0) continue;
    if (a.lse) {
      a.rows.row[row] = xent_row(target, a.lse[t], a.dloss[t]);
    } else {
      a.rows.target[row] = target;
    }
  }
  if (last == a.T && tid == 0) {
    a.rows.offsets[0] = 0;
    a.rows.offsets[1] = next;
  }
}

// Up to kXentGatherRows tokens: a wave numbers a token and copies 1024 columns of its row,
// in one launch (two launches: 9.4 us for 4.9, 104 tokens of H = 1399).
constexpr int kXentGatherRows = 1024, kXentGatherCols = 1024;

__global__ void __launch_bounds__(256) xent_gather_kernel(XentPlaceArgs a) {
  const int lane = (int)threadIdx.x & 63;
  const unsigned chunks = (unsigned)max((a.H + kXentGatherCols - 1) / kXentGatherCols, 1);
  const unsigned w = (unsigned)__builtin_amdgcn_readfirstlane(
      (int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
  const int t = (int)(w / chunks), chunk = (int)(w % chunks);
  if (t >= (int)a.T) return;
  const int target = a.targets.of(t);
  int row = 0;   // those before with a target; four rounds' loads, or all, in flight
  auto count = [&](auto from, auto to) {
    constexpr int I = decltype(from)::value, N = decltype(to)::value - I;
    int before[N];
#pragma unroll
    for (int i = 0; i < N; ++i) before[i] = a.targets.of(min((I + i) * 64 + lane, t));
#pragma unroll
    for (int i = 0; i < N; ++i)
      row += __popcll(__ballot(before[i] >= 0 && (I + i) * 64 + lane < t));
  };
  count(std::integral_constant<int, 0>(), std::integral_constant<int, 4>());
  if (t > 256)
    count(std::integral_constant<int, 4>(), std::integral_constant<int, kXentGatherRows / 64>());
  if (chunk == 0 && lane == 0) {
    a.rows.place[t] = target >= 0 ? row : -1;
    if (target >= 0) {
      if (a.lse) a.rows.row[row] = xent_row(target, a.lse[t], a.dloss[t]);
      else a.rows.target[row] = target;
    }
    if (t == (int)a.T - 1) {
      a.rows.offsets[0] = 0;
      a.rows.offsets[1] = row + (target >= 0 ? 1 : 0);
    }
  }
  if (target < 0) return;
  const int col = chunk * kXentGatherCols + 4 * lane;
  const float* const from = a.X + t * a.ldx + col;
  float* const to = a.rows.X + (int64_t)row * a.H + col;
  f32x4 v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (a.H - col > 256 * u) v[u] = load_upto(from + 256 * u, a.H - col - 256 * u);
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (a.H - col > 256 * u) store_upto(to + 256 * u, a.H - col - 256 * u, v[u]);
}

// A few tokens' rows as they stand; without a target a gradient of 0.
__global__ void __launch_bounds__(64) xent_rows_kernel(XentPlaceArgs a) {
  const int64_t t = threadIdx.x;
  if (t >= a.T) return;
  const int target = a.targets.of(t);
  XentRow row = {-1, 0.0f, 0.0f, 0.0f};
  if (target >= 0) row = xent_row(target, a.lse[t], a.dloss[t]);
  a.rows.row[t] = row;
}

// A wave takes 256 columns of a row of the planes, four a lane.
constexpr int kXentPlanesCols = 1024;   // of a workgroup

// Where this lane is: false, nowhere.  (A wave's lanes agree on the row.)
__device__ __forceinline__ bool xent_planes_at(const XentPlanesArgs& a, int& row, int& col) {
  const int blocks = (a.N + kXentPlanesCols - 1) / kXentPlanesCols;
  row = (int)(blockIdx.x / (unsigned)blocks);
  col = (int)(blockIdx.x % (unsigned)blocks) * kXentPlanesCols + 4 * (int)threadIdx.x;
  return col < a.N;
}
__device__ __forceinline__ f32x4 xent_planes_sum(const XentPlanesArgs& a, int row, int col) {
  constexpr int U = 8;   // planes in flight
  const int left = a.N - col;
  const int64_t plane = (int64_t)a.rows * a.N;
  const float* const p = a.planes + (int64_t)row * a.N + col;
  f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < a.count; s0 += U) {
    f32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s0 + u < a.count) v[u] = load_upto(p + (s0 + u) * plane, left);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s0 + u < a.count) z += v[u];
  }
  return z;
}

__global__ void __launch_bounds__(256) xent_planes_stats_kernel(XentPlanesArgs a) {
  int row, col;
  const bool in = xent_planes_at(a, row, col);
  const int target = a.targets.of(row);
  if (target < 0 || __ballot(in) == 0) return;   // whole waves
  f32x4 z = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  if (in) {
    const f32x4 v = xent_planes_sum(a, row, col);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (col + e < a.N) z[e] = v[e];
      if (col + e == target) a.hit[row] = v[e];   // a target is one of the columns
    }
  }
  float m = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
  for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float ref = xent_reference(m);
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) s += __builtin_amdgcn_exp2f(fmaf(z[e], kLog2e, -ref));
  s = sum64(s);
  if ((threadIdx.x & 63) != 0) return;
  const int64_t at = (int64_t)(col / 256) * a.rows + row;
  a.max[at] = m;
  a.sum[at] = s;
}

__global__ void __launch_bounds__(256) xent_planes_grad_kernel(XentPlanesArgs a) {
  int row, col;
  if (!xent_planes_at(a, row, col)) return;
  XentRow info;
  if (a.row) {
    if (row >= a.offsets[1]) return;
    info = a.row[row];
  } else {
    const int target = a.targets.of(row);
    if (target < 0) return;
    info = xent_row(target, a.lse[row], a.dloss[row]);
  }
  f32x4 z = xent_planes_sum(a, row, col);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float p = __builtin_amdgcn_exp2f(fmaf(z[e], kLog2e, -info.ref) - info.rest);
    z[e] = (p - (info.target - a.column0 == col + e ? 1.0f : 0.0f)) * info.grad;
  }
  store_upto(a.dZ + (int64_t)row * a.N + col, a.N - col, z);
}

// The strips of ROWS tokens' rows: part p of a token takes strips p, p + PARTS ..,
// sixteen at a time, and the parts meet by halves.  Many tokens: 32, which read whole
// cache lines (8192 tokens of 512 strips: 18 us with 16).
constexpr int kXentLossThreads = 1024;

template <int ROWS>
__global__ void __launch_bounds__(kXentLossThreads) xent_loss_kernel(XentLossArgs a) {
  constexpr int U = 16, PARTS = kXentLossThreads / ROWS;
  __shared__ float all_m[PARTS][ROWS], all_s[PARTS][ROWS];
  const int i = (int)threadIdx.x % ROWS, p = (int)threadIdx.x / ROWS;
  const int64_t t = (int64_t)blockIdx.x * ROWS + i;
  const bool kept = t < a.T && a.targets.of(t) >= 0;
  const int64_t row = !kept ? 0 : a.place ? a.place[t] : t;
  const float hit = kept && p == 0 ? a.hit[row] : 0.0f;
  float m = -INFINITY, s = 0.0f;   // the sum relative to m's reference
  if (kept) {
    for (int j0 = p; j0 < a.strips; j0 += U * PARTS) {
      float mm[U], ss[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * PARTS;
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
  for (int half = PARTS / 2; half > 0; half /= 2) {
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
