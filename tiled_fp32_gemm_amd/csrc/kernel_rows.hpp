// kernel_rows.hpp -- the epilogue products for a few rows (one token of a
// decoder, or an expert's few tokens): op(B) is read once, straight into
// registers, and multiplied with vector FMAs.
//
// Such a product is bound by reading B (2 R flop a float for R rows, where the
// chip has 32 flop for each float of HBM bandwidth), so what counts is bytes in
// flight: a workgroup of four or eight waves takes a few columns and splits K
// over its threads, each with several 16-byte groups in flight, and the partial
// sums meet once at the end, first within the waves, then through LDS in wave
// order.  No second launch and no workspace.  A (R rows) comes from the caches.
//
//   rows_fast_kernel   B is N x K: a wave takes four columns (four rows of B),
//                      its lanes 256 consecutive k at a time.  KW = 1: each of
//                      the four waves has columns of its own and all of K.
//                      KW = 4: they share the columns and take K by turns, for
//                      N too small to fill the chip otherwise.
//                      DEEP: more loads in flight, in more registers.
//   rows_slow_kernel   B is K x N: LC lanes take 4 LC consecutive columns of
//                      four consecutive k rows, the others further k.
//
// Measured on MI355X (B of 64 MiB, 4096 x 4096, from HBM, one row): fast 12.8 us
// (KW = 4 16.2), slow 18.2 us at 16 columns a workgroup and eight waves (four:
// 18.8; 32 columns 19.1, 64: 24.6, too few workgroups); product_kernel with its
// second launch takes 19.5 and 20.8 us.  11008 x 4096: fast 30.4 us (5.9 TB/s), slow
// 32.2 at 64 columns (four waves: 42.9; 32 columns 43.2).
//
// Fast, four rows: two steps in flight (DEEP) 13.1 us, one 15.2; eight rows: a
// step's loads before the other's products (DEEP) 16.5 us, one step at a time
// 17.9 (one to four rows that way: level or slower).  Over a short K the waves
// that the registers keep out cost more: 16 rows of eight groups, K = 1024, 24.2 us
// DEEP and 22.9; so DEEP is for K of 2048 and more.
//
// B is loaded nontemporal (one row by 4096 x 4096: 14.2 -> 12.7 us, 8192 x 8192:
// 45 -> 43 us, 6.2 TB/s), but for the slow kernel's narrow blocks, whose
// neighbours want the other half of a cache line (17.0 -> 18.3 us).
//
// Both take rows in chunks of R (more rows than R are further workgroups), of
// one product or of groups, and A stored M x K.
#pragma once

#include "kernel_product.hpp"

namespace sg {

constexpr int kRowsThreads = 256;

// Sums v[0 .. N-1] over the lanes of a wave that differ in bits D, D/2, ..,
// LAST: halves are exchanged while there are several values, so that a lane
// ends with N / (lanes summed) of them, v[0] on, or one.  Returns the number of
// the first.
template <int D, int LAST, int N, int V>
__device__ __forceinline__ int spread_sum(float (&v)[V], int lane) {
  if constexpr (D < LAST) {
    return 0;
  } else if constexpr (N > 1) {
    const bool up = (lane & D) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float give = up ? v[i] : v[i + N / 2];
      const float keep = up ? v[i + N / 2] : v[i];
      v[i] = keep + __shfl_xor(give, D);
    }
    return (up ? N / 2 : 0) + spread_sum<D / 2, LAST, N / 2, V>(v, lane);
  } else {
    v[0] += __shfl_xor(v[0], D);
    return spread_sum<D / 2, LAST, 1, V>(v, lane);
  }
}

// The chunk of rows and the block of columns of this workgroup.
struct RowsPlace {
  int row0, rows, group, block;
};

template <int R>
__device__ __forceinline__ bool rows_place(const ProductArgs& g, RowsPlace& p) {
  if (g.mode == kRowGroups) {
    RowTile t;
    if (!row_group_tile<R>(g, (int)threadIdx.x & 63, t)) return false;
    p.group = __builtin_amdgcn_readfirstlane(t.group);
    p.row0 = __builtin_amdgcn_readfirstlane(t.first + t.tm * R);
    p.rows = min(R, __builtin_amdgcn_readfirstlane(t.end) - p.row0);
    p.block = __builtin_amdgcn_readfirstlane(t.tn);
    return true;
  }
  int tm, tn;
  tile_order(xcd_order((int)blockIdx.x, (int)gridDim.x), g.tiles_m, g.tiles_n, g.group_m, tm, tn);
  p.group = 0;
  p.row0 = tm * R;
  p.rows = min(R, g.M - p.row0);
  p.block = tn;
  return true;
}

__device__ __forceinline__ void finish_one(const ProductArgs& g, const RowsPlace& p, int r, int col,
                                           float z) {
  const int64_t row = p.row0 + r;
  if (g.bias) z += g.bias[p.group * g.ld_bias + col];
  if (g.preact) g.preact[row * g.ldp + col] = z;
  with_activation(g.act, [&](auto which) { z = activate<decltype(which)::value>(z); });
  if (g.residual) z += g.residual[row * g.ldr + col];
  g.C[row * g.ldc + col] = z;
}

template <int R, int NC, int KW, bool DEEP>
__global__ void __launch_bounds__(kRowsThreads) rows_fast_kernel(ProductArgs g) {
  constexpr int V = R * NC;
  constexpr int STEP = 256 * KW;            // k taken at a time
  __shared__ float part[4][V];
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  RowsPlace p;
  if (!rows_place<R>(g, p)) return;
  // Waves that split k share their columns.
  const int n0 = (p.block * (4 / KW) + (KW == 4 ? 0 : wave)) * NC;
  const float* a[R];
  const float* b[NC];
  // Rows and columns past the end repeat the last one; their sums are dropped.
#pragma unroll
  for (int r = 0; r < R; ++r)
    a[r] = g.A + (int64_t)(p.row0 + min(r, p.rows - 1)) * g.lda;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    b[c] = (g.mode == kRowGroups ? g.B + p.group * g.stride_b : g.B) +
           (int64_t)min(n0 + c, g.N - 1) * g.ldb;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  auto take = [&](const f32x4 (&av)[R], const f32x4 (&bv)[NC]) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < NC; ++c)
          acc[r * NC + c] = fmaf(av[r][e], bv[c][e], acc[r * NC + c]);
  };
  int k = 4 * (KW == 4 ? (int)threadIdx.x : lane);
  if constexpr (DEEP && V > 16) {
    // Two steps' registers by turns: a step's loads go out before the other's
    // products.
    f32x4 av[2][R], bv[2][NC];
    auto load = [&](int s, int at) {
#pragma unroll
      for (int c = 0; c < NC; ++c) bv[s][c] = load_upto_once(b[c] + at, 4);
#pragma unroll
      for (int r = 0; r < R; ++r) av[s][r] = *reinterpret_cast<const f32x4u*>(a[r] + at);
    };
    if (k + 4 <= g.K) load(0, k);
    while (k + 4 <= g.K) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s == 1 && k + 4 > g.K) break;
        if (k + STEP + 4 <= g.K) load(1 - s, k + STEP);
        __builtin_amdgcn_sched_barrier(0);
        take(av[s], bv[s]);
        k += STEP;
      }
    }
  } else {
    constexpr int U = V < 16 || (DEEP && V == 16) ? 2 : 1;   // steps in flight
    for (; k + (U - 1) * STEP + 4 <= g.K; k += U * STEP) {
      f32x4 av[U][R], bv[U][NC];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
          bv[u][c] = load_upto_once(b[c] + k + u * STEP, 4);
#pragma unroll
        for (int r = 0; r < R; ++r)
          av[u][r] = *reinterpret_cast<const f32x4u*>(a[r] + k + u * STEP);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) take(av[u], bv[u]);
    }
  }
  for (; k < g.K; k += STEP) {
    f32x4 av[R], bv[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) bv[c] = load_upto(b[c] + k, g.K - k);
#pragma unroll
    for (int r = 0; r < R; ++r) av[r] = load_upto(a[r] + k, g.K - k);
    take(av, bv);
  }
  const int which = spread_sum<32, 1, V, V>(acc, lane);
  // Lanes that share a value hold it alike.
  if ((lane & (64 / V - 1)) == 0) part[wave][which] = acc[0];
  __syncthreads();
  const int i = KW == 4 ? (int)threadIdx.x : lane;
  if (i >= V) return;
  const int r = i / NC, col = n0 + i % NC;
  if (r < p.rows && col < g.N)
    finish_one(g, p, r, col,
               KW == 4 ? ((part[0][i] + part[1][i]) + part[2][i]) + part[3][i] : part[wave][i]);
}

template <int R, int LC, int T>
__global__ void __launch_bounds__(T) rows_slow_kernel(ProductArgs g) {
  constexpr int V = 4 * R;
  constexpr int KR = T / LC;   // groups of four k rows at a time
  constexpr int SHARE = 64 / LC;          // of them in a wave
  constexpr int LEFT = V > SHARE ? V / SHARE : 1;   // values a lane ends with
  __shared__ float part[T / 64][V * LC];
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  RowsPlace p;
  if (!rows_place<R>(g, p)) return;
  const int cg = tid % LC;
  const int n0 = p.block * 4 * LC;
  const int col = n0 + 4 * cg, left = g.N - col;
  const float* a[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    a[r] = g.A + (int64_t)(p.row0 + min(r, p.rows - 1)) * g.lda;
  const float* const b = (g.mode == kRowGroups ? g.B + p.group * g.stride_b : g.B) + col;
  float acc[V];   // [row][column]
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  auto sweep = [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    auto load = [&](int k) {
      const float* const p = b + (int64_t)k * g.ldb;
      if (!kWhole) return load_upto(p, left);
      return LC == 16 ? load_upto_once(p, 4) : load_upto(p, 4);
    };
    constexpr int kFlight = 2;   // groups of rows in flight
    int k = 4 * (tid / LC);
#pragma unroll kFlight
    for (; k + 4 <= g.K; k += 4 * KR) {
      f32x4 av[R], bv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) bv[e] = load(k + e);
#pragma unroll
      for (int r = 0; r < R; ++r) av[r] = *reinterpret_cast<const f32x4u*>(a[r] + k);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            acc[r * 4 + c] = fmaf(av[r][e], bv[e][c], acc[r * 4 + c]);
    }
    for (; k < g.K; ++k) {   // the last, partial group of four: one thread's
      const f32x4 bv = load(k);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r * 4 + c] = fmaf(a[r][k], bv[c], acc[r * 4 + c]);
    }
  };
  if (left >= 4) sweep(std::true_type());
  else if (left > 0) sweep(std::false_type());
  // Over the wave's SHARE lanes of a column group.
  const int first = spread_sum<32, LC, V, V>(acc, lane);
  if (V >= SHARE || lane / LC % (SHARE / V > 0 ? SHARE / V : 1) == 0) {
#pragma unroll
    for (int i = 0; i < LEFT; ++i) {   // [row][column], as they are read below
      const int v = first + i;
      part[wave][v / 4 * (4 * LC) + 4 * cg + v % 4] = acc[i];
    }
  }
  __syncthreads();
  for (int i = tid; i < V * LC; i += T) {
    // Consecutive threads take consecutive columns of a row.
    const int r = i / (4 * LC), c = i % (4 * LC);
    if (r < p.rows && n0 + c < g.N) {
      float z = part[0][i];
#pragma unroll
      for (int w = 1; w < T / 64; ++w) z += part[w][i];
      finish_one(g, p, r, n0 + c, z);
    }
  }
}

}  // namespace sg
