// kernel_act_backward.hpp -- dZ = dC * act'(Z) with the column sums of dZ (the
// bias gradient), over all rows or per group of rows.
//
// One pass: a workgroup takes 256 columns of one strip of a group's rows, each
// wave every fourth row, four columns a lane; the waves' sums are added in
// wave order through LDS and go to the strip's row of W, or straight to the
// result when a group is one strip.  column_sum_kernel adds the strips in
// order.  Bound by HBM: dC and Z are read once and dZ is written once.
//
// Loads and stores are 16 bytes at any 4-byte alignment (global, not buffer,
// accesses); only a row's last one to three columns go one by one.
#pragma once

#include "activation.hpp"
#include "product_args.hpp"
#include "rows.hpp"

namespace sg {

struct ActBackwardArgs {
  const float* dC;
  const float* Z;       // null: act is NONE
  float* dZ;            // null: only the sums
  float* dbias;         // null: no sums
  float* W;             // [strip][group][N], when strips > 1
  int64_t lddc, ldz, lddz, lddb;
  const int32_t* offsets;   // null: one group of all rows
  int M, N, groups, strips, act;
  int blocks_n;         // ceil(N / kActCols)
};

constexpr int kActCols = 256;
constexpr int kActWaves = 4;

template <bool HAS_Z>
__global__ void __launch_bounds__(64 * kActWaves) act_backward_kernel(ActBackwardArgs a) {
  __shared__ f32x4 part[kActWaves][64];
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  int w = (int)blockIdx.x;
  const int bn = w % a.blocks_n;
  w /= a.blocks_n;
  const int strip = w % a.strips, group = w / a.strips;
  int begin = 0, end = a.M;
  if (a.offsets) group_range(a.offsets, group, a.M, begin, end);
  const int per = (int)(((int64_t)(end - begin) + a.strips - 1) / a.strips);
  const int r0 = (int)min((int64_t)begin + (int64_t)strip * per, (int64_t)end);
  const int r1 = (int)min((int64_t)r0 + per, (int64_t)end);
  const int col = bn * kActCols + 4 * lane, left = a.N - col;
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  if (left > 0) {
    constexpr int U = 4;   // rows in flight
    for (int r = r0 + wave; r < r1; r += U * kActWaves) {
      f32x4 d[U], z[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = r + u * kActWaves;
        if (row < r1) {
          d[u] = load_upto(a.dC + row * a.lddc + col, left);
          if constexpr (HAS_Z) z[u] = load_upto(a.Z + row * a.ldz + col, left);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = r + u * kActWaves;
        if (row < r1) {
          if constexpr (HAS_Z) {
#pragma unroll
            for (int e = 0; e < 4; ++e) d[u][e] *= activation_slope(a.act, z[u][e]);
          }
          if (a.dZ) store_upto(a.dZ + row * a.lddz + col, left, d[u]);
          sum += d[u];
        }
      }
    }
  }
  if (!a.dbias) return;
  part[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || left <= 0) return;
#pragma unroll
  for (int q = 1; q < kActWaves; ++q) sum += part[q][lane];
  float* out = a.strips > 1 ? a.W + ((int64_t)strip * a.groups + group) * a.N + col
                            : a.dbias + group * a.lddb + col;
  store_upto(out, left, sum);
}

// dbias[g][j] = sum over s of W[s][g][j], for 64 columns a workgroup: each
// wave adds a quarter of the strips, then the quarters are added in order.
__global__ void __launch_bounds__(256) column_sum_kernel(ActBackwardArgs a) {
  __shared__ float part[4][64];
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  const int blocks = (a.N + 63) / 64;
  const int group = (int)blockIdx.x / blocks;
  const int col = ((int)blockIdx.x - group * blocks) * 64 + lane;
  const int64_t plane = (int64_t)a.groups * a.N;
  const int per = (a.strips + 3) / 4;
  const int s1 = min((wave + 1) * per, a.strips);
  float sum = 0.0f;
  if (col < a.N) {
    const float* p = a.W + (int64_t)group * a.N + col;
#pragma unroll 8
    for (int s = wave * per; s < s1; ++s) sum += p[s * plane];
  }
  part[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || col >= a.N) return;
  a.dbias[group * a.lddb + col] = ((sum + part[1][lane]) + part[2][lane]) + part[3][lane];
}

}  // namespace sg
