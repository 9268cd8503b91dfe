// kernel_act_backward.hpp -- dZ = dC * act'(Z) with the column sums of dZ (the
// bias gradient), over all rows or per group of rows.
//
// One pass: the rows are cut into spans (a group's last one shorter, an empty
// group's only one empty), and a workgroup of four waves takes a span and up to
// 256 columns, four columns a lane.  Narrow matrices put several rows side by
// side in a wave (lpr lanes a row).  A span's sums are added through LDS in a
// fixed order and go to its row of W, or straight to the result when it is the
// group's only one; column_sum_kernel adds the rows of W in a fixed order.  Without
// room for W the same pass makes dZ, and act_sum_kernel adds the spans up by
// itself, sixteen columns a workgroup, in the same order: the sums go by the sizes
// alone, whatever room there is.
//
// Bound by HBM: dC and Z are read once and dZ is written once.  Measured on
// MI355X with SILU or GELU: 65536 x 128 in 18.8 us (5.3 TB/s), 4096 x 4096 in 38 to
// 41 us (5 TB/s), and 4.7 us for the spans' sums; both passes over 16384 x 2048 of 64
// groups 79 us, of one group with all the rows and 63 without 81 (as many spans
// for every group: 101 and 878), of 16384 x 1024 of 1000 groups, where every wave
// has many to count, 59 (38 and 1690).  The loads are nontemporal, which
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
  float* W;             // [span][N], of the groups with several; null: no room
  int64_t lddc, ldz, lddz, lddb;
  const int32_t* offsets;   // null: one group of all rows
  int M, N, groups;
  int span, spans;      // rows of a span; how many there are room for
  int lpr;              // lanes along a row: 1, 2, 4 .. 64
  int blocks_n;         // ceil(N / (4 lpr))
};

constexpr int kActWaves = 4;
// A lane's sum starts anew after so many rows: its rounding errors grow with
// n / 256 + 256 rather than n.
constexpr int kActRun = 256;

// A group's rows and spans.
struct ActGroup {
  int begin, end;
  int first, count;   // its spans
};

// The group of span `at` (SPAN), or number `at` of the groups with several spans;
// false: there is none.  Every wave counts the groups' spans for itself: up to 64
// groups one a lane, more of them first several a lane and then that lane's.
template <bool SPAN>
__device__ __forceinline__ bool act_group(const ActBackwardArgs& a, int at, int& group,
                                          ActGroup& out) {
  if (!a.offsets) {
    group = 0;
    out = {0, a.M, 0, a.spans};
    return true;
  }
  const int lane = (int)threadIdx.x & 63;
  int b, e, n;
  auto count = [&](int g) {   // without a branch, so that several groups' loads go out together
    group_range(a.offsets, min(g, a.groups - 1), a.M, b, e);
    n = g < a.groups ? max(1, (int)(((unsigned)(e - b) + (unsigned)a.span - 1) / (unsigned)a.span))
                     : 0;
  };
  auto key = [&]() { return SPAN ? n : n > 1 ? 1 : 0; };
  int base = 0, width = 64, before = 0, spans = 0;   // of the groups before base
  if (a.groups > 64) {
    width = (a.groups + 63) / 64;
    int keys = 0, all = 0;
#pragma unroll 8
    for (int i = 0; i < width; ++i) {
      count(lane * width + i);
      keys += key();
      all += n;
    }
    const int upto = scan64(keys);
    const uint64_t hit = __ballot(upto > at);
    if (hit == 0) return false;
    const int h = __ffsll((unsigned long long)hit) - 1;
    base = h * width;
    before = __builtin_amdgcn_readlane(upto - keys, h);
    spans = SPAN ? before : __builtin_amdgcn_readlane(scan64(all) - all, h);
  }
  count(lane < width ? base + lane : a.groups);
  const int upto = before + scan64(key());
  const uint64_t hit = __ballot(upto > at);
  if (hit == 0) return false;
  const int h = __ffsll((unsigned long long)hit) - 1;
  group = base + h;
  out.begin = __builtin_amdgcn_readlane(b, h);
  out.end = __builtin_amdgcn_readlane(e, h);
  out.count = __builtin_amdgcn_readlane(n, h);
  out.first = spans + __builtin_amdgcn_readlane(SPAN ? upto - before : scan64(n), h) - out.count;
  // Offsets that fall describe more spans than there are, or make their number
  // overflow.
  return SPAN ? (unsigned)(at - out.first) < (unsigned)out.count
              : out.first >= 0 && out.first < a.spans;
}

// dZ (if it is wanted) and this lane's sum over rows r, r + beside .. below end.
template <int ACT>
__device__ __forceinline__ f32x4 act_rows(const ActBackwardArgs& a, int64_t r, int64_t end,
                                          int beside, int col, int left, float* dZ) {
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f}, total = sum;
  constexpr int U = 4;   // rounds of rows in flight
  int run = 0;
  for (; r < end; r += U * beside) {
    f32x4 d[U], z[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = r + u * beside;
      if (row < end) {
        d[u] = load_upto_once(a.dC + row * a.lddc + col, left);
        if constexpr (ACT != SGEMM_ACT_NONE) z[u] = load_upto_once(a.Z + row * a.ldz + col, left);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = r + u * beside;
      if (row < end) {
        if constexpr (ACT != SGEMM_ACT_NONE) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = d[u][e] * activation_slope<ACT>(z[u][e]);
            asm("" : "+v"(v));   // summed as it is stored, not in one FMA
            d[u][e] = v;
          }
        }
        if (dZ) store_upto(dZ + row * a.lddz + col, left, d[u]);
        sum += d[u];
      }
    }
    if (++run == kActRun / U) {
      total += sum;
      sum = {0.0f, 0.0f, 0.0f, 0.0f};
      run = 0;
    }
  }
  return total + sum;
}

template <int ACT>
__global__ void __launch_bounds__(64 * kActWaves) act_backward_kernel(ActBackwardArgs a) {
  __shared__ f32x4 part[kActWaves * 64];
  const int lane = (int)threadIdx.x & 63;
  const int bn = (int)blockIdx.x % a.blocks_n, span = (int)blockIdx.x / a.blocks_n;
  int group;
  ActGroup g;
  if (!act_group<true>(a, span, group, g)) return;
  const bool later = g.count > 1 && !a.W;   // act_sum_kernel's sums
  if (later && !a.dZ) return;
  const int64_t r0 = g.begin + (int64_t)(span - g.first) * a.span;
  const int64_t r1 = min(r0 + a.span, (int64_t)g.end);
  const int beside = 64 / a.lpr * kActWaves;   // rows at a time
  const int col = 4 * (bn * a.lpr + lane % a.lpr), left = a.N - col;
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  if (left > 0) sum = act_rows<ACT>(a, r0 + (int)threadIdx.x / a.lpr, r1, beside, col, left, a.dZ);
  if (!a.dbias || later) return;
  part[threadIdx.x] = sum;
  __syncthreads();
  if ((int)threadIdx.x >= a.lpr || left <= 0) return;
  for (int q = 1; q < beside; ++q) sum += part[q * a.lpr + lane];
  float* out = g.count > 1 ? a.W + (int64_t)span * a.N + col : a.dbias + group * a.lddb + col;
  store_upto(out, left, sum);
}

// dbias of the groups with several spans: the sum over their rows of W, COLS
// columns and a group a workgroup.  Span s is in part s mod 64; the parts, each
// added in order, meet by halves.  A thread has every T-th part, so that any COLS
// gives the same sum: 16 where that leaves few workgroups, 128 where it makes many
// short ones.
constexpr int kSumParts = 64;

template <int COLS>
constexpr int kSumThreads = COLS == 16 ? 1024 : 256;

template <int COLS>
__global__ void __launch_bounds__(kSumThreads<COLS>) column_sum_kernel(ActBackwardArgs a) {
  constexpr int NT = kSumThreads<COLS>, T = NT / COLS, MINE = kSumParts / T;
  __shared__ float part[NT];
  const int tid = (int)threadIdx.x;
  const int blocks = (a.N + COLS - 1) / COLS;
  int group = (int)blockIdx.x / blocks;
  const int col = ((int)blockIdx.x - group * blocks) * COLS + tid % COLS;
  ActGroup g;
  if (!act_group<false>(a, group, group, g)) return;
  const int count = min(g.count, a.spans - g.first);
  float sum[MINE];
#pragma unroll
  for (int i = 0; i < MINE; ++i) sum[i] = 0.0f;
  if (col < a.N) {
    const float* p = a.W + (int64_t)g.first * a.N + col;
    if constexpr (MINE == 1) {
#pragma unroll 8
      for (int s = tid / COLS; s < count; s += kSumParts) sum[0] += p[(int64_t)s * a.N];
    } else {
      for (int s0 = tid / COLS; s0 < count; s0 += kSumParts) {
        float v[MINE];
#pragma unroll
        for (int i = 0; i < MINE; ++i) v[i] = p[(int64_t)min(s0 + i * T, count - 1) * a.N];
#pragma unroll
        for (int i = 0; i < MINE; ++i) sum[i] += s0 + i * T < count ? v[i] : 0.0f;
      }
    }
  }
#pragma unroll
  for (int half = MINE / 2; half > 0; half /= 2)
#pragma unroll
    for (int i = 0; i < half; ++i) sum[i] += sum[i + half];
  part[tid] = sum[0];
  for (int half = NT / 2; half >= COLS; half /= 2) {
    __syncthreads();
    if (tid < half) part[tid] += part[tid + half];
  }
  if (tid < COLS && col < a.N) a.dbias[group * a.lddb + col] = part[tid];
}

// The same without W: a group and up to 16 columns a workgroup, which takes as many
// spans at a time as its threads have room for and adds them up as the two kernels
// above do.  With dZ made before it, it reads that (as dC).  Bound by the loads in
// flight of few workgroups: 65536 x 128 (eight) 208 us, 4096 x 4096 25, 1000 x 777 7,
// against the 5 of the pass through W.
template <int ACT>
__global__ void __launch_bounds__(1024) act_sum_kernel(ActBackwardArgs a) {
  constexpr int NT = 1024;
  __shared__ f32x4 part[NT];
  __shared__ f32x4 acc[kSumParts * 4];         // [part][column]
  const int tid = (int)threadIdx.x;
  const int L = min(a.lpr, 4);                 // lanes along a row
  const int beside = 64 / a.lpr * kActWaves;   // rows of a span at a time
  const int P = NT / L / beside;               // spans at a time: 4 .. 64
  const int blocks = (a.N + 4 * L - 1) / (4 * L);
  int group = (int)blockIdx.x / blocks;
  const int bn = (int)blockIdx.x - group * blocks;
  ActGroup g;
  if (!act_group<false>(a, group, group, g)) return;
  const int q0 = tid / L % beside, j = tid / L / beside;
  const int col = 4 * (bn * L + tid % L), left = a.N - col;
  if (tid < kSumParts * L) acc[tid] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < g.count; s0 += P) {
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t r0 = g.begin + (int64_t)(s0 + j) * a.span;
    if (left > 0)
      sum = act_rows<ACT>(a, r0 + q0, min(r0 + a.span, (int64_t)g.end), beside, col, left, nullptr);
    part[tid] = sum;
    __syncthreads();
    // P divides kSumParts, so a thread meets its own words of acc only.
    const int s = s0 + tid / L;
    if (tid < P * L && s < g.count) {
      const f32x4* p = part + tid / L * beside * L + tid % L;
      f32x4 v = p[0];
      for (int q = 1; q < beside; ++q) v += p[q * L];
      acc[s % kSumParts * L + tid % L] += v;
    }
    __syncthreads();
  }
  for (int half = kSumParts / 2 * L; half >= L; half /= 2) {
    if (tid < half) acc[tid] += acc[tid + half];
    __syncthreads();
  }
  if (tid < L && left > 0) store_upto(a.dbias + group * a.lddb + col, left, acc[tid]);
}

}  // namespace sg
