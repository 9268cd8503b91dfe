// kernel_xent_few.hpp -- both gradients of the cross entropy over a product for up to
// sixteen rows.
//
//   dB = sum over tokens of x by dz        dX = dz·op(B)'
//
// Each entry of B meets the entry of dB at its place: a lane holds a few columns of the
// rows of the one factor (X, or dz) in registers, goes down B's rows with the other
// factor's numbers from LDS, and for each row stores dB and takes B into its part of
// dX.  B is read and dB written once, which is what it is bound by; the parts of dX
// are added up by xent_few_sum_kernel.  Rows without a target count as zeros, so
// nothing has to be copied together for so few.  (dz comes from the logits, a launch
// before this one that reads B too: twice in all.)
//
//   xent_few_down_kernel    B is V x H: a lane has four columns of H, two for sixteen rows,
//                           in each of four waves, which take the rows by turns; dX's
//                           sums stay in registers.
//                           Without the gradients: the logits where B is H x V.
//   xent_few_across_kernel  B is H x V: a wave has 256 of V, four waves side by side;
//                           a row of B is summed over the lanes, several rows at once.
//
// Measured on MI355X (us; tokens, H, V; the kernel's average over thirty passes and three
// weights in turn):
//   down    8, 3264, 7145  35.9 (5.2 TB/s), 7, 3271, 7145  41, 4, 1024, 33000  46.0
//           (5.9), 4, 1030, 33000  57.5, 1, 2885, 29858  155 (4.4), 16, 1024, 32768  61
//           (4.4); the logits of 8, 1024, 32768  30.0 (4.5) and 2, 2871, 34831  74 (5.4),
//           where products by rows or tiles took 87 to 180
//   across  8, 1024, 32768  49.7 (5.4), 2, 2871, 34831  164 (4.9), 16, 1024, 32768  65 (4.2)
//   All of the gradients, calls one after another with three weights in turn, against the
//   rows' copies, three products and dX's scatter: down, sixteen rows 1024, 32768  92 for
//   111, 64, 60000  30 for 41 (four columns in a lane would spill: 185 for 113), 12, 2217,
//   5372  51 for 66; across, 9, 1030, 20001  64 for 96, sixteen rows 1024, 32768  92 for 114
//   (85 with one weight, as some of it stays in the caches)
//   Columns four together in a lane (16-byte accesses at any alignment) down: 3271 59.5,
//   1030 87.  dB past the caches down: 49 and 76, as the ends of unaligned rows' pieces
//   are then written in parts; across, where a workgroup's piece is 4 KB, in them: 149 for
//   163, but the next reading of B 111 for 74.  The logits' reading of B past the caches:
//   the gradients 75 for 55 (8, 1024, 32768).
#pragma once

#include "kernel_rows.hpp"
#include "xent_args.hpp"

namespace sg {

constexpr int kXentFewThreads = 256;
constexpr int kXentFewAcross = 64;   // most rows of B of a workgroup across

// A lane's C columns of a block of 64 C: from `first` on, 64 apart, and never past the
// last, which is repeated there (its sums are dropped), as loads that some lanes leave out
// are waited for one by one.  Rows begin at scalar addresses, so these are all that is
// held of one.
template <int C>
struct FewCols {
  unsigned at[C];   // bytes
  int left;         // columns from `first` on

  __device__ __forceinline__ FewCols(int first, int cols) : left(cols - first) {
#pragma unroll
    for (int e = 0; e < C; ++e) at[e] = 4u * (unsigned)min(first + 64 * e, cols - 1);
  }
  template <bool ONCE>
  __device__ __forceinline__ void load(const float* row, float (&v)[C]) const {
#pragma unroll
    for (int e = 0; e < C; ++e) {
      const char* const at_e = reinterpret_cast<const char*>(row) + at[e];
      const float* const p = reinterpret_cast<const float*>(at_e);
      v[e] = ONCE ? __builtin_nontemporal_load(p) : *p;
    }
  }
  __device__ __forceinline__ void store(float* row, const float (&v)[C]) const {
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (64 * e < left) *reinterpret_cast<float*>(reinterpret_cast<char*>(row) + at[e]) = v[e];
  }
};

// Columns of a lane down: two for sixteen rows, whose factors and sums would spill.
constexpr int xent_few_cols(int R) { return R <= 8 ? 4 : 2; }

// The tokens with a target, a bit each.
__device__ __forceinline__ unsigned xent_few_kept(const XentFewArgs& a) {
  const int lane = (int)threadIdx.x & 63;
  return (unsigned)__ballot(lane < a.T && a.targets.of(lane < a.T ? lane : 0) >= 0);
}

template <int R, bool GRAD>
__global__ void __launch_bounds__(kXentFewThreads) xent_few_down_kernel(XentFewArgs a) {
  constexpr int U = 8;                 // rows of B in flight
  constexpr int C = xent_few_cols(R);
  constexpr int CHUNK = 128, NUMBERS = CHUNK * R;
  __shared__ __attribute__((aligned(16))) float room[2 * R * 64 * C];   // numbers, then sums
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned place = (unsigned)xcd_order((int)blockIdx.x, (int)gridDim.x);
  const int block = (int)(place % (unsigned)a.blocks), part = (int)(place / (unsigned)a.blocks);
  const int first = part * a.part, last = min(first + a.part, a.rows);
  const FewCols<C> cols(block * (64 * C) + lane, a.cols);
  const unsigned kept = xent_few_kept(a);
  float q[R][C], acc[R][C];
#pragma unroll
  for (int t = 0; t < R; ++t) {
#pragma unroll
    for (int e = 0; e < C; ++e) q[t][e] = acc[t][e] = 0.0f;
    if (GRAD && (kept >> t & 1)) cols.template load<false>(a.Q + (int64_t)t * a.ldq, q[t]);
  }
  for (int c0 = first; c0 < last; c0 += CHUNK) {
    const int rows = min(CHUNK, last - c0);
    if (c0 > first) __syncthreads();
    for (int i = tid; i < NUMBERS; i += kXentFewThreads) {   // [row][token]
      const int r = i % CHUNK, t = i / CHUNK;
      room[r * R + t] = r < rows && (kept >> t & 1) ? a.P[(int64_t)t * a.ldp + c0 + r] : 0.0f;
    }
    __syncthreads();
    const float* const b = a.B + (int64_t)c0 * a.ldb;
    float* const d = a.D + (int64_t)c0 * a.ldd;
    auto load = [&](int r, float (&v)[C]) {
      cols.template load<GRAD>(b + (int64_t)r * a.ldb, v);
    };
    auto take = [&](int r, const float (&v)[C]) {
      float g[C] = {};
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const float p = room[r * R + t];
#pragma unroll
        for (int e = 0; e < C; ++e) {
          acc[t][e] = fmaf(p, v[e], acc[t][e]);
          if (GRAD) g[e] = fmaf(p, q[t][e], g[e]);
        }
      }
      if (GRAD && a.D) cols.store(d + (int64_t)r * a.ldd, g);
    };
    for (int r0 = wave * U; r0 < rows; r0 += 4 * U) {
      if (r0 + U <= rows) {
        float v[U][C];
#pragma unroll
        for (int u = 0; u < U; ++u) load(r0 + u, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) take(r0 + u, v[u]);
      } else {
        for (int r = r0; r < rows; ++r) {
          float v[C];
          load(r, v);
          take(r, v);
        }
      }
    }
  }
  if (a.planes == nullptr) return;
  // The four waves' sums, by halves.
  typedef float part_t __attribute__((ext_vector_type(C)));
  part_t* const join = reinterpret_cast<part_t*>(room);
#pragma unroll
  for (int half = 2; half > 0; half /= 2) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int t = 0; t < R; ++t) {
        part_t p;
#pragma unroll
        for (int e = 0; e < C; ++e) p[e] = acc[t][e];
        join[((wave - half) * R + t) * 64 + lane] = p;
      }
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const part_t p = join[(wave * R + t) * 64 + lane];
#pragma unroll
        for (int e = 0; e < C; ++e) acc[t][e] += p[e];
      }
    }
  }
  if (wave > 0) return;
#pragma unroll
  for (int t = 0; t < R; ++t)
    if (t < a.T) cols.store(a.planes + ((int64_t)part * a.T + t) * a.cols, acc[t]);
}

template <int R>
__global__ void __launch_bounds__(kXentFewThreads, R <= 8 ? 4 : 2)
    xent_few_across_kernel(XentFewArgs a) {
  constexpr int U = R <= 4 ? 8 : 4;    // rows of B in flight
  constexpr int S = U * R;                   // sums over the lanes at once
  constexpr int ROWS = kXentFewAcross;
  __shared__ __attribute__((aligned(16))) float numbers[ROWS * R];   // [row][token]
  __shared__ float sum[4][ROWS * R];
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned place = blockIdx.x;
  const int block = (int)(place % (unsigned)a.blocks);
  const int first = (int)(place / (unsigned)a.blocks) * a.part;
  const int rows = min(a.part, a.rows - first);
  const int col = block * 1024 + 4 * tid, left = a.cols - col;
  const unsigned kept = xent_few_kept(a);
  f32x4 q[R];
#pragma unroll
  for (int t = 0; t < R; ++t) {
    q[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if ((kept >> t & 1) && left > 0) q[t] = load_upto(a.Q + (int64_t)t * a.ldq + col, left);
  }
  for (int i = tid; i < ROWS * R; i += kXentFewThreads) {
    const int r = i % ROWS, t = i / ROWS;
    numbers[r * R + t] = r < rows && (kept >> t & 1) ? a.P[(int64_t)t * a.ldp + first + r] : 0.0f;
  }
  __syncthreads();
  const float* const b = a.B + (int64_t)first * a.ldb + col;
  float* const d = a.D + (int64_t)first * a.ldd + col;
  // All of a wave's lanes take part in its sums, whatever columns they have.
  auto sweep = [&](auto all) {
    constexpr bool kAll = decltype(all)::value;
    const int n = kAll ? 4 : left;
    for (int r0 = 0; r0 < rows; r0 += U) {
      f32x4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float* const at = b + (int64_t)min(r0 + u, rows - 1) * a.ldb;
        if (kAll) {
          v[u] = load_upto(at, 4);
        } else {   // no load is left out, as it would be waited for
#pragma unroll
          for (int e = 0; e < 4; ++e) v[u][e] = at[min(e, n - 1)];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[u][e] = e < n ? v[u][e] : 0.0f;
        }
      }
      float s[S];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        f32x4 g = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const float p = numbers[(r0 + u) * R + t];
          float dot = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dot = fmaf(v[u][e], q[t][e], dot);
            g[e] = fmaf(p, q[t][e], g[e]);
          }
          s[u * R + t] = dot;
        }
        if (a.D && n > 0 && r0 + u < rows) store_upto_once(d + (int64_t)(r0 + u) * a.ldd, n, g);
      }
      const int which = spread_sum<32, 1, S, S>(s, lane);
      if ((lane & (64 / S - 1)) == 0) sum[wave][r0 * R + which] = s[0];
    }
  };
  if (block * 1024 + 256 * wave + 256 <= a.cols) sweep(std::true_type());
  else sweep(std::false_type());
  if (a.planes == nullptr) return;
  __syncthreads();
  for (int i = tid; i < ROWS * a.T; i += kXentFewThreads) {
    const int r = i % ROWS, t = i / ROWS, at = r * R + t;
    if (r < rows)
      a.planes[((int64_t)block * a.T + t) * a.rows + first + r] =
          ((sum[0][at] + sum[1][at]) + sum[2][at]) + sum[3][at];
  }
}

// dX of its planes: four lanes take sixteen columns of a token, 64 times, each every
// 64th plane.
constexpr int kXentFewSumCols = 16;

__global__ void __launch_bounds__(kXentFewThreads) xent_few_sum_kernel(XentFewSumArgs a) {
  constexpr int U = 4;   // planes in flight
  __shared__ f32x4 share[64][4];
  const int tid = (int)threadIdx.x, lane = tid & 3, p = tid >> 2;
  const int blocks = (a.H + kXentFewSumCols - 1) / kXentFewSumCols;
  const int t = (int)(blockIdx.x / (unsigned)blocks);
  const int col = (int)(blockIdx.x % (unsigned)blocks) * kXentFewSumCols + 4 * lane;
  const int left = a.H - col;
  f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t plane = (int64_t)a.T * a.H;
  if (left > 0 && a.targets.of(t) >= 0) {
    const float* const at = a.planes + (int64_t)t * a.H + col;
    for (int s0 = p; s0 < a.count; s0 += 64 * U) {
      f32x4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s0 + 64 * u < a.count) v[u] = load_upto(at + (s0 + 64 * u) * plane, left);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s0 + 64 * u < a.count) z += v[u];
    }
  }
  share[p][lane] = z;
  for (int half = 32; half > 0; half /= 2) {
    __syncthreads();
    if (p < half) share[p][lane] = z += share[p + half][lane];
  }
  if (p == 0 && left > 0) store_upto(a.dX + t * a.lddx + col, left, z);
}

}  // namespace sg
