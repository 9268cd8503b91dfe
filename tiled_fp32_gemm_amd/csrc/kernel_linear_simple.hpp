// kernel_linear_simple.hpp -- the epilogue products in their simplest form:
// 16 x 16 tiles, one output per thread.
#pragma once

#include "activation.hpp"
#include "product_args.hpp"

namespace sg {

template <bool TA, bool TB>
__global__ void __launch_bounds__(256) product_simple_kernel(ProductArgs g) {
  constexpr int T = 16;
  __shared__ float As[T][T + 1], Bs[T][T + 1];
  int tile = (int)blockIdx.x, group = 0, m0 = 0, m_end = g.M, k_begin = 0, k_end = g.K;
  int tn = 0;
  if (g.mode == kRowGroups) {
    tn = tile % g.tiles_n;
    int t = tile / g.tiles_n;
    bool found = false;
    for (; group < g.groups; ++group) {
      int b, e;
      group_range(g.offsets, group, g.rows, b, e);
      const int tiles = (e - b + T - 1) / T;
      if (t < tiles) {
        m0 = b + t * T;
        m_end = e;
        found = true;
        break;
      }
      t -= tiles;
    }
    if (!found) return;
  } else {
    const int tiles = g.tiles_m * g.tiles_n;
    group = tile / tiles;
    tile -= group * tiles;
    tn = tile % g.tiles_n;
    m0 = (tile / g.tiles_n) * T;
    if (g.mode == kSumGroups) group_range(g.offsets, group, g.rows, k_begin, k_end);
  }
  const int n0 = tn * T;
  const int x = (int)threadIdx.x & 15, y = (int)threadIdx.x >> 4;
  const float* B = g.mode == kRowGroups ? g.B + group * g.stride_b : g.B;
  float acc = 0.0f;
  for (int k0 = k_begin; k0 < k_end; k0 += T) {
    const int am = m0 + y, ak = k0 + x, bk = k0 + y, bn = n0 + x;
    As[y][x] = am < m_end && ak < k_end
                   ? g.A[TA ? (int64_t)ak * g.lda + am : (int64_t)am * g.lda + ak] : 0.0f;
    Bs[y][x] = bk < k_end && bn < g.N
                   ? B[TB ? (int64_t)bn * g.ldb + bk : (int64_t)bk * g.ldb + bn] : 0.0f;
    __syncthreads();
    for (int k = 0; k < T; ++k) acc = fmaf(As[y][k], Bs[k][x], acc);
    __syncthreads();
  }
  const int m = m0 + y, n = n0 + x;
  if (m >= m_end || n >= g.N) return;
  float z = acc;
  if (g.bias) z += g.bias[(g.mode == kRowGroups ? group * g.ld_bias : 0) + n];
  if (g.preact) g.preact[(int64_t)m * g.ldp + n] = z;
  float v = activate(g.act, z);
  if (g.residual) v += g.residual[(int64_t)m * g.ldr + n];
  float* C = g.mode == kSumGroups ? g.C + group * g.stride_c : g.C;
  C[(int64_t)m * g.ldc + n] = v;
}

}  // namespace sg
