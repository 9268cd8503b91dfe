// kernel_route.hpp -- a router's scores to each token's experts and their
// weights, and the gradient of the weights.
//
// G lanes of a wave share a token, V groups of four experts each, so that the
// logits are read once, 16 bytes a lane.  A lane packs each expert's score and
// number into one double whose order is that of (score, lowest number first):
// the score's bits made monotonic, then 2047 less the expert, under a fixed
// exponent.  Then a comparison of two experts is v_max_f64 and v_min_f64.  A lane
// sorts its experts K at a time (Batcher's odd-even mergesort), keeps the best K,
// and the lanes' lists meet by a butterfly: the larger of A[i] and B[K-1-i] are
// the best K of both, a bitonic sequence, which log2 K rounds sort.
//
// The choice is that of exact scores.  Without a bias, and without groups that
// count two scores, it goes by the logits themselves, whose order is the scores'.
// Otherwise FP32 scores decide unless two that matter are closer than their
// errors (near() below); then the wave computes that token's scores and choice
// again in FP64 (refine), which happens to one token in some hundreds.
#pragma once

#include "../../include/sgemm_moe.h"
#include "activation.hpp"
#include "lanes.hpp"
#include "rows.hpp"

namespace sg {

constexpr int kRouteTop = SGEMM_MOE_MAX_TOP;

struct RouteArgs {
  const float* logits;
  const float* bias;     // null: none
  int32_t* experts;
  float* weights;
  const float* dweights;   // backward
  float* dlogits;
  int64_t ld, ldd, T;
  int E, top, scoring, renormalize;
  int groups, top_groups, group_best;
  int size, per;         // experts of a group; 2^20 / size, rounded up
  float scale;
};

// The group of an expert, without a division: exact below 1024.
__device__ __forceinline__ int group_of(const RouteArgs& a, int expert) {
  return (int)((uint32_t)expert * (uint32_t)a.per >> 20);
}

// Lane exchange within groups of G lanes: step s of the butterfly.  The mirrors
// stand for xor 4 and xor 8, as the lanes of a quad (of eight) agree by then.
template <int STEP>
__device__ __forceinline__ int exchanged(int v) {
  static_assert(STEP >= 0 && STEP <= 4, "up to 32 lanes");
  constexpr int ctrl = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140;
  if constexpr (STEP == 4) return __shfl_xor(v, 16);
  return __builtin_amdgcn_update_dpp(0, v, ctrl, 0xF, 0xF, true);
}
template <int STEP>
__device__ __forceinline__ float exchanged(float v) {
  return __builtin_bit_cast(float, exchanged<STEP>(__builtin_bit_cast(int, v)));
}
template <int STEP>
__device__ __forceinline__ double exchanged(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)exchanged<STEP>((int)(uint32_t)b);
  const uint32_t hi = (uint32_t)exchanged<STEP>((int)(uint32_t)(b >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// f(integral_constant<int, step>) for the steps of G lanes.
template <int G, class F>
__device__ __forceinline__ void butterfly(F f) {
  f(std::integral_constant<int, 0>());
  f(std::integral_constant<int, 1>());
  if constexpr (G >= 8) f(std::integral_constant<int, 2>());
  if constexpr (G >= 16) f(std::integral_constant<int, 3>());
  if constexpr (G >= 32) f(std::integral_constant<int, 4>());
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  butterfly<G>([&](auto s) { v += exchanged<decltype(s)::value>(v); });
  return v;
}
template <int G>
__device__ __forceinline__ int group_sum(int v) {
  butterfly<G>([&](auto s) { v += exchanged<decltype(s)::value>(v); });
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  butterfly<G>([&](auto s) { v = fmaxf(v, exchanged<decltype(s)::value>(v)); });
  return v;
}

// A float's bits as an unsigned number of the same order; NaN is infinity, and -0
// is 0.  0 is no float's: an expert that cannot be chosen.
__device__ __forceinline__ uint32_t ordered(float f) {
  f = f != f ? INFINITY : f + 0.0f;
  const uint32_t b = __builtin_bit_cast(uint32_t, f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __builtin_bit_cast(float, k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}

__device__ __forceinline__ double packed(uint32_t key, int expert) {
  const uint32_t hi = key >> 21 | 0x40000000u, lo = key << 11 | (uint32_t)(2047 - expert);
  return key == 0u ? 0.0 : __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// -1: none.
__device__ __forceinline__ int packed_expert(double d) {
  const uint64_t b = __builtin_bit_cast(uint64_t, d);
  return b == 0 ? -1 : 2047 - (int)((uint32_t)b & 2047u);
}
__device__ __forceinline__ float packed_score(double d) {
  const uint64_t b = __builtin_bit_cast(uint64_t, d);
  return unordered((uint32_t)(b >> 11));
}

__device__ __forceinline__ void larger_first(double& a, double& b) {
  const double hi = __builtin_fmax(a, b);
  b = __builtin_fmin(a, b);
  a = hi;
}

// Batcher's odd-even mergesort, largest first.
template <int N>
__device__ __forceinline__ void sort_down(double (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p))
            larger_first(v[i + j], v[i + j + k]);
}

// The best N of two lists of N, largest first.
template <int N>
__device__ __forceinline__ void merge_down(double (&a)[N], const double (&b)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = __builtin_fmax(a[i], b[N - 1 - i]);
#pragma unroll
  for (int k = N / 2; k >= 1; k /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & k) == 0) larger_first(a[i], a[i + k]);
}

// This wave's own LDS: its writes before, its reads after.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ bool choosable(double v) { return !(v == -(double)INFINITY); }

// One token's choice from scores in FP64, by a whole wave; `score` has room for E.
__device__ __forceinline__ void refine(const RouteArgs& a, int64_t t, double* score, int* ids) {
  const int lane = (int)threadIdx.x & 63;
  const float* const row = a.logits + t * a.ld;
  const double none = -(double)INFINITY;
  double top = none, sum = 0.0;
  if (a.scoring == SGEMM_SCORE_SOFTMAX) {
    for (int e = lane; e < a.E; e += 64) top = fmax(top, (double)row[e]);
    for (int d = 32; d > 0; d >>= 1) top = fmax(top, __shfl_xor(top, d));
    for (int e = lane; e < a.E; e += 64) sum += exp((double)row[e] - top);
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  }
  for (int e = lane; e < a.E; e += 64) {
    const double x = (double)row[e];
    double c = a.scoring == SGEMM_SCORE_SOFTMAX ? exp(x - top) / sum : 1.0 / (1.0 + exp(-x));
    if (a.bias) c += (double)a.bias[e];
    score[e] = !choosable(x) ? none : c != c ? (double)INFINITY : c;
  }
  wave_lds_fence();
  uint32_t stays = ~0u;
  if (a.groups > 1) {
    double best = none, second = none;
    if (lane < a.groups)
      for (int e = lane * a.size; e < (lane + 1) * a.size; ++e) {
        const double v = score[e];
        second = fmax(second, fmin(v, best));
        best = fmax(best, v);
      }
    if (a.group_best == 2 && choosable(second)) best += second;
    int rank = 0;
    for (int q = 0; q < a.groups; ++q) {
      const double other = __shfl(best, q);
      rank += other > best || (other == best && q < lane) ? 1 : 0;
    }
    stays = (uint32_t)__ballot(lane < a.groups && rank < a.top_groups);
  }
  for (int j = 0; j < a.top; ++j) {
    double best = none;
    int at = a.E;
    for (int e = lane; e < a.E; e += 64) {
      const double v = score[e];
      if (v > best && (stays >> group_of(a, e) & 1)) {
        best = v;
        at = e;
      }
    }
    for (int d = 32; d > 0; d >>= 1) {
      const double v = __shfl_xor(best, d);
      const int e = __shfl_xor(at, d);
      if (v > best || (v == best && e < at)) {
        best = v;
        at = e;
      }
    }
    if (lane == 0) {
      ids[j] = at < a.E ? at : -1;
      if (at < a.E) score[at] = none;
    }
    wave_lds_fence();
  }
}

// What FP32 scores may be off, in half steps of 2^-24.  exp_accurate and the
// reciprocal are within 8 of their value, a softmax's exponent adds its own
// distance from the largest (0.37 of the largest score at most) and the sum of
// the exponentials 28 (13 additions in a row, 8 of each term, ln E of the
// exponents), which all scores share but which moves them against the bias.  Two
// such errors, rounded up; beside them the addition of the bias rounds once.
constexpr float kHalfStep = 5.9604645e-8f;
constexpr float kSoftmaxOff = 96.0f * kHalfStep, kSigmoidOff = 24.0f * kHalfStep;

template <int G, int V, int K>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs a) {
  constexpr int TOKENS = 256 / G, N = 4 * V;
  // Each wave has its tokens' part of both.
  __shared__ __attribute__((aligned(16))) uint32_t keys[TOKENS * N * G];
  __shared__ int ids[TOKENS][kRouteTop];
  static_assert(64 / G * N * G * 4 >= N * G * 8, "a wave's keys hold one token's FP64 scores");
  const int lane = (int)threadIdx.x & 63, g = (int)threadIdx.x % G;
  const int sub = (int)threadIdx.x / G;
  const int64_t t0 = (int64_t)blockIdx.x * TOKENS + sub;
  const bool live = t0 < a.T;
  const int64_t t = live ? t0 : a.T - 1;
  const float* const row = a.logits + t * a.ld;
  const bool by_score = a.bias || (a.groups > 1 && a.group_best > 1);
  const bool whole = a.scoring == SGEMM_SCORE_SOFTMAX && (by_score || !a.renormalize);

  float c[N];   // the logits, then what the choice goes by
  bool can[N];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = 4 * (g + i * G), left = a.E - col;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (left > 0) v = load_upto(row + col, left);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[4 * i + e] = v[e];
      can[4 * i + e] = e < left && !(v[e] == -INFINITY);
    }
  }
  float top = -INFINITY, inv = 1.0f;   // of the whole softmax
  float off = kSigmoidOff;
  if (whole) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (can[i]) top = fmaxf(top, c[i]);
    top = group_max<G>(top);
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float p = exp_accurate(c[i] - top);
      if (by_score) c[i] = p;
      if (can[i]) sum[i & 3] += p;
    }
    inv = 1.0f / group_sum<G>((sum[0] + sum[1]) + (sum[2] + sum[3]));
    off = kSoftmaxOff * inv;
  }
  if (by_score) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = 4 * (g + i * G), left = a.E - col;
      f32x4 b = {0.0f, 0.0f, 0.0f, 0.0f};
      if (a.bias && left > 0) b = load_upto(a.bias + col, left);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float s = whole ? c[4 * i + e] * inv : sigmoid(c[4 * i + e]);
        c[4 * i + e] = s + b[e];
        can[4 * i + e] = can[4 * i + e] && !(c[4 * i + e] == -INFINITY);
      }
    }
  }
  // Whether two scores are too near each other to tell which is larger.
  auto near = [&](float x, float y) {
    return x - y <= off + 2.0f * kHalfStep * (fabsf(x) + fabsf(y));
  };
  bool unsure = false;

  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = can[i] ? ordered(c[i]) : 0u;
  if (a.groups > 1) {
    // Lane g looks at groups g, g + G ..: the best and second best of each, then
    // how many groups come before it.
    uint32_t* const mine = keys + sub * (N * G);
    const int size = a.size;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = key[4 * i + e];
      *reinterpret_cast<u32x4*>(mine + 4 * (g + i * G)) = v;
    }
    wave_lds_fence();
    constexpr int ROUNDS = (SGEMM_MOE_MAX_GROUPS + G - 1) / G;
    uint32_t total[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const int q = r * G + g;
      total[r] = 0u;
      if (r * G < a.groups && q < a.groups) {
        uint32_t best = 0u, second = 0u;
        int at = g % size;   // neighbouring groups may begin on the same bank
        for (int i = 0; i < size; ++i) {
          const uint32_t k = mine[q * size + at];
          at = at + 1 == size ? 0 : at + 1;
          second = max(second, min(k, best));
          best = max(best, k);
        }
        total[r] = a.group_best == 2 && second != 0u
                       ? ordered(unordered(best) + unordered(second)) : best;
      }
    }
    wave_lds_fence();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
      if (r * G < a.groups && r * G + g < a.groups) mine[r * G + g] = total[r];
    wave_lds_fence();
    uint32_t stays = 0;
    uint32_t last = 0u, next = 0u;   // the last group that stays, the first that does not
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      if (r * G < a.groups) {
        const int q = r * G + g;
        int rank = q < a.groups ? 0 : a.groups;
        for (int o = 0; o < a.groups; ++o) {
          const uint32_t other = mine[o];
          rank += other > total[r] || (other == total[r] && o < q) ? 1 : 0;
        }
        if (rank == a.top_groups - 1) last = total[r];
        if (rank == a.top_groups) next = total[r];
        const uint64_t bits = __ballot(rank < a.top_groups) >> (lane - g);
        stays |= (uint32_t)(bits & ((uint64_t(1) << G) - 1)) << (r * G);
      }
    }
    if (by_score && a.top_groups < a.groups) {
      butterfly<G>([&](auto s) {
        last = max(last, (uint32_t)exchanged<decltype(s)::value>((int)last));
        next = max(next, (uint32_t)exchanged<decltype(s)::value>((int)next));
      });
      // Two scores a group: twice the errors.
      if (next != 0u) {
        const float x = unordered(last), y = unordered(next);
        unsure = x - y <= 2.0f * off + 8.0f * kHalfStep * (fabsf(x) + fabsf(y));
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = 4 * (g + (i >> 2) * G) + (i & 3);
      if (e < a.E && !(stays >> group_of(a, e) & 1)) key[i] = 0u;
    }
  }

  // This lane's best K, then all lanes'.
  double best[K];
#pragma unroll
  for (int j = 0; j < K; ++j) best[j] = 0.0;
#pragma unroll
  for (int i0 = 0; i0 < N; i0 += K) {
    double v[K];
#pragma unroll
    for (int j = 0; j < K; ++j)
      v[j] = i0 + j < N ? packed(key[i0 + j < N ? i0 + j : 0],
                                 4 * (g + ((i0 + j) >> 2) * G) + ((i0 + j) & 3))
                        : 0.0;
    sort_down(v);
    if (i0 == 0) {
#pragma unroll
      for (int j = 0; j < K; ++j) best[j] = v[j];
    } else {
      merge_down(best, v);
    }
  }
  butterfly<G>([&](auto s) {
    double other[K];
#pragma unroll
    for (int j = 0; j < K; ++j) other[j] = exchanged<decltype(s)::value>(best[j]);
    merge_down(best, other);
  });
#pragma unroll
  for (int j = 0; j < K; ++j)
    if (j % G == g && j < a.top) ids[sub][j] = packed_expert(best[j]);

  if (by_score) {
    float least = -INFINITY;   // the last one chosen
    bool full = false;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (j + 1 < K && j + 1 < a.top && packed_expert(best[j + 1 < K ? j + 1 : 0]) >= 0 &&
          near(packed_score(best[j]), packed_score(best[j + 1 < K ? j + 1 : 0])))
        unsure = true;
      if (j == a.top - 1 && packed_expert(best[j]) >= 0) {
        least = packed_score(best[j]);
        full = true;
      }
    }
    // No other may be near the last one.
    int close = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      close += key[i] != 0u && near(least, unordered(key[i])) ? 1 : 0;
    close = group_sum<G>(close);
    if (full && close > a.top) unsure = true;
    uint64_t again = __ballot(unsure && live);
    double* const room = reinterpret_cast<double*>(keys + (sub - lane / G) * (N * G));
    wave_lds_fence();
    while (again != 0) {
      const int first = __ffsll((unsigned long long)again) - 1;
      const int of = first / G;   // of the wave's tokens
      const int64_t token = (int64_t)blockIdx.x * TOKENS + (sub - lane / G) + of;
      refine(a, token, room, ids[sub - lane / G + of]);
      again &= ~(((uint64_t(1) << G) - 1) << (of * G));
    }
  }
  wave_lds_fence();

  // Weights: lane g those of choices g, g + G ..
  constexpr int J = (K + G - 1) / G;
  int id[J];
  float l[J], w[J], most = -INFINITY, total = 0.0f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    id[j] = j * G + g < a.top ? ids[sub][j * G + g] : -1;
    l[j] = id[j] >= 0 ? row[id[j]] : -INFINITY;
    most = fmaxf(most, l[j]);
  }
  if (a.renormalize) {
    // Relative to the largest of the chosen, so that no sum vanishes.
    most = group_max<G>(most);
    if (a.scoring == SGEMM_SCORE_SIGMOID) most = fminf(most, 0.0f);
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (a.scoring == SGEMM_SCORE_SOFTMAX)
      w[j] = exp_accurate(l[j] - (a.renormalize ? most : top)) * inv;
    else if (!a.renormalize || l[j] > 0.0f)
      w[j] = sigmoid(l[j]);
    else
      w[j] = exp_accurate(l[j] - most) / (1.0f + exp_accurate(l[j]));
    if (id[j] < 0) w[j] = 0.0f;
    total += w[j];
  }
  if (a.renormalize) total = group_sum<G>(total);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int at = j * G + g;
    if (!live || at >= a.top) continue;
    a.experts[t * a.top + at] = id[j];
    a.weights[t * a.top + at] =
        id[j] < 0 ? 0.0f : a.renormalize ? w[j] / total * a.scale : w[j] * a.scale;
  }
}

// dlogits from dweights.  A token's row is made in LDS: zeros, the chosen experts'
// values (lane g's choices g, g + G ..; equal ids share their sum), then read back
// four columns a lane, where a whole softmax adds its common term.
template <int G, int V>
__global__ void __launch_bounds__(256) route_backward_kernel(RouteArgs a) {
  constexpr int TOKENS = 256 / G, N = 4 * V, J = (kRouteTop + G - 1) / G;
  __shared__ __attribute__((aligned(16))) float rows[TOKENS * N * G];
  __shared__ int ids[TOKENS][kRouteTop];
  __shared__ float values[TOKENS][kRouteTop];
  const int g = (int)threadIdx.x % G, sub = (int)threadIdx.x / G;
  const int64_t t0 = (int64_t)blockIdx.x * TOKENS + sub;
  const bool live = t0 < a.T;
  const int64_t t = live ? t0 : a.T - 1;
  const float* const row = a.logits + t * a.ld;
  const bool whole = a.scoring == SGEMM_SCORE_SOFTMAX && !a.renormalize;
  float* const mine = rows + sub * (N * G);
  f32x4 p[V];
  float top = -INFINITY, inv = 0.0f;
  if (whole) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = 4 * (g + i * G), left = a.E - col;
      p[i] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (left > 0) {
        const f32x4 v = load_upto(row + col, left);
#pragma unroll
        for (int e = 0; e < 4; ++e) p[i][e] = e < left ? v[e] : -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, p[i][e]);
    }
    top = group_max<G>(top);
    // A token without any expert to choose has no gradient.
    const float from = top == -INFINITY ? 0.0f : top;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) p[i][e] = exp_accurate(p[i][e] - from);
      sum += p[i];
    }
    const float total = group_sum<G>((sum[0] + sum[1]) + (sum[2] + sum[3]));
    inv = total == 0.0f ? 0.0f : 1.0f / total;
    top = from;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    *reinterpret_cast<f32x4*>(mine + 4 * (g + i * G)) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // The chosen experts' own terms.
  int id[J];
  float v[J], w[J], dot = 0.0f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int at = j * G + g;
    id[j] = -1;
    v[j] = w[j] = 0.0f;
    if (at < a.top) {
      id[j] = a.experts[t * a.top + at];
      if (id[j] >= a.E) id[j] = -1;
      if (id[j] >= 0) {
        v[j] = a.dweights[t * a.top + at];
        if (a.renormalize) w[j] = a.weights[t * a.top + at];
        else if (whole) w[j] = exp_accurate(row[id[j]] - top) * inv * a.scale;
      }
    }
    dot += v[j] * w[j];
  }
  if (a.renormalize || whole) dot = group_sum<G>(dot);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int at = j * G + g;
    if (a.renormalize)
      v[j] = w[j] * (v[j] - dot / a.scale);
    else
      v[j] *= a.scale;
    if (a.scoring == SGEMM_SCORE_SIGMOID && id[j] >= 0) {
      float rest;
      const float s = sigmoid_both(row[id[j]], rest);
      v[j] *= a.renormalize ? rest : s * rest;
    }
    if (at < a.top) {
      ids[sub][at] = id[j];
      values[sub][at] = v[j];
    }
  }
  wave_lds_fence();
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (id[j] < 0) continue;
    float sum = 0.0f;
    for (int o = 0; o < a.top; ++o)
      if (ids[sub][o] == id[j]) sum += values[sub][o];
    mine[id[j]] = sum;
  }
  wave_lds_fence();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = 4 * (g + i * G), left = a.E - col;
    f32x4 d = *reinterpret_cast<const f32x4*>(mine + col);
    if (whole) d = p[i] * inv * (d - dot);
    if (live && left > 0) store_upto(a.dlogits + t * a.ldd + col, left, d);
  }
}

}  // namespace sg
