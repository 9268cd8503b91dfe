// kernel_product_reduce.hpp -- the second pass of a split product: the splits'
// partial sums added in split order, then the epilogue.
//
// W holds `splits` planes of `rows` x N floats.  A 64-thread workgroup takes 256
// columns of one row, a thread four of them, eight splits' loads in flight.
// kRowGroups: rows of no group are left alone, a row's group is found by
// halving.  kSumGroups: a plane holds the groups' matrices one after another.
// Bound by HBM and by its launch: (splits + 1 + residual + preact) M N 4 bytes;
// 5.8 us for four splits of 1024 x 1024 (21 MB), 5.1 us for 32 of 256 x 128.
// Sharing a row's planes among four waves instead took 16.7 and 6.0 us (four
// times the waves to launch).
#pragma once

#include "activation.hpp"
#include "product_args.hpp"
#include "rows.hpp"

namespace sg {

constexpr int kProductReduceCols = 256;

__global__ void __launch_bounds__(64) product_reduce_kernel(ProductArgs g) {
  const int chunks = (g.N + kProductReduceCols - 1) / kProductReduceCols;
  const int64_t wide = (int64_t)blockIdx.x / chunks;
  const int col = ((int)blockIdx.x - (int)wide * chunks) * kProductReduceCols +
                  4 * (int)threadIdx.x;
  const int left = g.N - col;
  int row = (int)wide, group = 0;
  const int64_t plane = (int64_t)g.M * g.N * (g.mode == kSumGroups ? g.groups : 1);
  float* C = g.C;
  if (g.mode == kSumGroups) {
    group = row / g.M;
    row -= group * g.M;
    C += group * g.stride_c;
  } else if (g.mode == kRowGroups) {
    // The last group that begins at or before the row (empty ones share their
    // beginning with the one after).
    int lo = 0, hi = g.groups;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (g.offsets[mid] <= row) lo = mid + 1;
      else hi = mid;
    }
    group = lo - 1;
    if (group < 0) return;
    int b, e;
    group_range(g.offsets, group, g.rows, b, e);
    if (row < b || row >= e) return;
  }
  if (left <= 0) return;
  const float* w = g.W + wide * g.N + col;
  constexpr int kBatch = 8;
  f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < g.splits; s0 += kBatch) {
    f32x4 v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (s0 + j < g.splits) v[j] = load_upto(w + (s0 + j) * plane, left);
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (s0 + j < g.splits) z += v[j];
  }
  if (g.bias) z += load_upto(g.bias + group * g.ld_bias + col, left);
  if (g.preact) store_upto(g.preact + (int64_t)row * g.ldp + col, left, z);
  with_activation(g.act, [&](auto which) {
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = activate<decltype(which)::value>(z[e]);
  });
  if (g.residual) z += load_upto(g.residual + (int64_t)row * g.ldr + col, left);
  store_upto(C + (int64_t)row * g.ldc + col, left, z);
}

}  // namespace sg
