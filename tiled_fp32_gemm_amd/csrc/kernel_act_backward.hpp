// kernel_act_backward.hpp -- dZ = dC * act'(Z) with the column sums of dZ (the
// bias gradient), over all rows or per group of rows.
//
// One pass: a workgroup of four waves takes a strip of a group's rows and up to
// 256 columns, four columns a lane.  Narrow matrices put several rows side by
// side in a wave (lpr lanes a row).  The sums are added through LDS in a fixed
// order and go to the strip's row of W, or straight to the result when a group
// is one strip; column_sum_kernel adds the strips in a fixed order.  Bound by
// HBM: dC and Z are read once and dZ is written once.  Measured on MI355X with
// SILU or GELU: 65536 x 128 in 18.6 us (5.4 TB/s), 4096 x 4096 in 41 us
// (4.9 TB/s), and 4.7 us for the strips' sums.  The loads are nontemporal, which
// leaves dZ in the caches for the products after it (41 instead of 45 us here,
// 109 -> 100 us with two products at K = 64).
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
  int M, N, groups, strips;
  int lpr;              // lanes along a row: 1, 2, 4 .. 64
  int blocks_n;         // ceil(N / (4 lpr))
};

constexpr int kActWaves = 4;

template <int ACT>
__global__ void __launch_bounds__(64 * kActWaves) act_backward_kernel(ActBackwardArgs a) {
  __shared__ f32x4 part[kActWaves * 64];
  const int lane = (int)threadIdx.x & 63;
  int w = (int)blockIdx.x;
  const int bn = w % a.blocks_n;
  w /= a.blocks_n;
  const int strip = w % a.strips, group = w / a.strips;
  int begin = 0, end = a.M;
  if (a.offsets) group_range(a.offsets, group, a.M, begin, end);
  const int per = (int)(((int64_t)(end - begin) + a.strips - 1) / a.strips);
  const int r0 = (int)min((int64_t)begin + (int64_t)strip * per, (int64_t)end);
  const int r1 = (int)min((int64_t)r0 + per, (int64_t)end);
  const int beside = 64 / a.lpr * kActWaves;   // rows at a time
  const int col = 4 * (bn * a.lpr + lane % a.lpr), left = a.N - col;
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  if (left > 0) {
    constexpr int U = 4;   // rounds of rows in flight
    for (int64_t r = r0 + (int)threadIdx.x / a.lpr; r < r1; r += U * beside) {
      f32x4 d[U], z[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = r + u * beside;
        if (row < r1) {
          d[u] = load_upto_once(a.dC + row * a.lddc + col, left);
          if constexpr (ACT != SGEMM_ACT_NONE) z[u] = load_upto_once(a.Z + row * a.ldz + col, left);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = r + u * beside;
        if (row < r1) {
          if constexpr (ACT != SGEMM_ACT_NONE) {
#pragma unroll
            for (int e = 0; e < 4; ++e) d[u][e] *= activation_slope<ACT>(z[u][e]);
          }
          if (a.dZ) store_upto(a.dZ + row * a.lddz + col, left, d[u]);
          sum += d[u];
        }
      }
    }
  }
  if (!a.dbias) return;
  part[threadIdx.x] = sum;
  __syncthreads();
  if ((int)threadIdx.x >= a.lpr || left <= 0) return;
  for (int q = 1; q < beside; ++q) sum += part[q * a.lpr + lane];
  float* out = a.strips > 1 ? a.W + ((int64_t)strip * a.groups + group) * a.N + col
                            : a.dbias + group * a.lddb + col;
  store_upto(out, left, sum);
}

// dbias[g][j] = sum over s of W[s][g][j], for kSumCols columns a workgroup:
// every 64th strip a thread, then the threads' sums by halves.
constexpr int kSumCols = 16;

__global__ void __launch_bounds__(1024) column_sum_kernel(ActBackwardArgs a) {
  __shared__ float part[1024];
  const int tid = (int)threadIdx.x;
  const int blocks = (a.N + kSumCols - 1) / kSumCols;
  const int group = (int)blockIdx.x / blocks;
  const int col = ((int)blockIdx.x - group * blocks) * kSumCols + tid % kSumCols;
  const int64_t plane = (int64_t)a.groups * a.N;
  float sum = 0.0f;
  if (col < a.N) {
    const float* p = a.W + (int64_t)group * a.N + col;
#pragma unroll 8
    for (int s = tid / kSumCols; s < a.strips; s += 1024 / kSumCols) sum += p[s * plane];
  }
  part[tid] = sum;
  for (int half = 512; half >= kSumCols; half /= 2) {
    __syncthreads();
    if (tid < half) part[tid] += part[tid + half];
  }
  if (tid < kSumCols && col < a.N) a.dbias[group * a.lddb + col] = part[tid];
}

}  // namespace sg
