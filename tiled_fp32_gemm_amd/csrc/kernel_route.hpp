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
// The choice is that of FP64 scores.  Without a bias, and without groups that
// count two scores, it goes by the logits themselves, whose order is the scores'.
// Otherwise FP32 scores decide unless two that matter are closer than their
// errors (kSoftmaxOff below, and each score's rounding at its own size, also where a
// group's two cancel), as for one token in about a thousand; then the wave
// computes the scores again in FP64, those that may be chosen (reorder), or all
// where the groups are open or there are too many (refine).
//
// Bound by vector instructions, 1357 a wave for eight tokens' best 8 of 256 in groups by
// sigmoid and bias, where the copies of 32768 such rows would take 7.3 us.  Measured on
// MI355X, calls one after another over several inputs: 16.3 to 19.5 us, by the inputs (2.5 of
// it the FP64 of the last waves); without bias and groups 10 to 11.5, 8191 tokens of 64
// experts 3.8.  Where the groups that stay have at most half of the experts, only those are sorted
// (all: 300 instructions and 1.1 us more).  Sixteen lanes a token instead of eight (twice
// the waves, half the experts a lane) took 23.9 for 19.9, a branch for each expert's special
// cases 37.  A batch of equal scores, all in FP64: 64 us, 78 in groups.
// The gradient is bound by HBM: 32768 x 256 (69 MB) with the whole softmax in 14.3 us (the
// kernel 16.4 on average of forty under the profiler, 13.9 at least); renormalised 9.0, by
// sigmoid 10.1 to 10.5 (33.6 MB to write, a cache line to read for each choice).
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
  return (int)(__umul24((uint32_t)expert, (uint32_t)a.per) >> 20);
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
// is 0.  An expert that cannot be chosen has -infinity's, which is the least.
__device__ __forceinline__ uint32_t ordered_bits(float f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t ordered(float f) {
  return ordered_bits(fminf(f, INFINITY) + 0.0f);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __builtin_bit_cast(float, k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}
constexpr uint32_t kNever = 0x007FFFFFu;   // ordered(-INFINITY)

__device__ __forceinline__ double packed(uint32_t key, int expert) {
  const uint32_t hi = __builtin_amdgcn_alignbit(0x200u, key, 21);   // an exponent before it
  const uint32_t lo = key << 11 | (uint32_t)(2047 - expert);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ uint32_t packed_key(double d) {
  return (uint32_t)(__builtin_bit_cast(uint64_t, d) >> 11);
}
// -1: none (0.0 is a place of a list that is not full).
__device__ __forceinline__ int packed_expert(double d) {
  return packed_key(d) <= kNever ? -1
                                 : 2047 - (int)((uint32_t)__builtin_bit_cast(uint64_t, d) & 2047u);
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

// Over a whole wave, all lanes with the same bits.
template <class F>
__device__ __forceinline__ double over_wave(double v, F f) {
  butterfly<16>([&](auto s) { v = f(v, exchanged<decltype(s)::value>(v)); });
  auto of = [&](int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  };
  return f(f(of(0), of(16)), f(of(32), of(48)));
}

// A token's scores in FP64, by a whole wave: `top` and `sum` of its softmax.
struct Exact {
  double top, sum;

  template <int Q>
  __device__ __forceinline__ void prepare(const RouteArgs& a, const float* row) {
    top = sum = 0.0;
    if (a.scoring != SGEMM_SCORE_SOFTMAX) return;
    const int lane = (int)threadIdx.x & 63;
    double l[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
      l[q] = lane + 64 * q < a.E ? (double)row[lane + 64 * q] : -(double)INFINITY;
    top = l[0];
#pragma unroll
    for (int q = 1; q < Q; ++q) top = fmax(top, l[q]);
    top = over_wave(top, [](double x, double y) { return fmax(x, y); });
#pragma unroll
    for (int q = 0; q < Q; ++q) sum += exp(l[q] - top);
    sum = over_wave(sum, [](double x, double y) { return x + y; });
  }
  // What an expert is chosen by; -infinity: not to be chosen.
  __device__ __forceinline__ double of(const RouteArgs& a, const float* row, int e) const {
    const double l = (double)row[e], b = a.bias ? (double)a.bias[e] : 0.0;
    const double s = (a.scoring == SGEMM_SCORE_SOFTMAX ? exp(l - top) / sum
                                                       : 1.0 / (1.0 + exp(-l))) + b;
    return l == -(double)INFINITY ? l : s != s ? (double)INFINITY : s;
  }
};

// The two ways back for a token that FP32 leaves open, each by a whole wave.  A
// launch ends with a wave that is here, so their chains are short.
//
// The order of `n` candidates, one a lane, among which the choice is.
template <int Q>
__device__ __forceinline__ void reorder(const RouteArgs& a, int64_t t, const int* list, int n,
                                        int* ids) {
  const int lane = (int)threadIdx.x & 63;
  const float* const row = a.logits + t * a.ld;
  const int e = lane < n ? list[lane] : 0;
  Exact exact;
  exact.prepare<Q>(a, row);
  const double c = exact.of(a, row, e);
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const double other = __shfl(c, i);
    const int o = __shfl(e, i);
    rank += other > c || (other == c && o < e) ? 1 : 0;
  }
  if (lane < n && rank < a.top) ids[rank] = e;
}

// The whole choice; Q experts a lane, `room` for all of them.
template <int Q>
__device__ __forceinline__ void refine(const RouteArgs& a, int64_t t, double* room, int* ids) {
  const int lane = (int)threadIdx.x & 63;
  const float* const row = a.logits + t * a.ld;
  const double none = -(double)INFINITY;
  Exact exact;
  exact.prepare<Q>(a, row);
  double c[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q)
    c[q] = lane + 64 * q < a.E ? exact.of(a, row, lane + 64 * q) : none;
  if (a.groups > 1) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (lane + 64 * q < a.E) room[lane + 64 * q] = c[q];
    wave_lds_fence();
    double best = none, second = none;
    if (lane < a.groups) {
#pragma unroll 8
      for (int i = 0; i < a.size; ++i) {
        const double v = room[lane * a.size + i];
        second = fmax(second, fmin(v, best));
        best = fmax(best, v);
      }
    }
    if (a.group_best == 2 && second != none) best += second;
    int rank = 0;
    for (int q = 0; q < a.groups; ++q) {
      const double other = __shfl(best, q);
      rank += other > best || (other == best && q < lane) ? 1 : 0;
    }
    const uint32_t stays = (uint32_t)__ballot(lane < a.groups && rank < a.top_groups);
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (!(stays >> group_of(a, min(lane + 64 * q, a.E - 1)) & 1)) c[q] = none;
    wave_lds_fence();   // `room` is read before another token's scores
  }
  for (int j = 0; j < a.top; ++j) {
    double best = c[0];
#pragma unroll
    for (int q = 1; q < Q; ++q) best = fmax(best, c[q]);
    best = over_wave(best, [](double x, double y) { return fmax(x, y); });
    int at = -1;
    if (best != none) {
#pragma unroll
      for (int q = Q - 1; q >= 0; --q) {
        const uint64_t hit = __ballot(c[q] == best);
        if (hit != 0) at = 64 * q + __ffsll((unsigned long long)hit) - 1;
      }
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (at == lane + 64 * q) c[q] = none;
    }
    if (lane == 0) ids[j] = at;
  }
}

// What FP32 scores may be off, in half steps of 2^-24.  quick_exp(x) is within 2 +
// 1.3 |x| of its value (the product rounds, and so does log2 e).
//   sigmoid  s (1 - s) (2 + 1.3 |x|) <= 0.8, and three more of s: 4
//   softmax  d from the largest, which rounds too: s (2 + 2.3 d) <= 2.85 of the
//            largest score; the sum of the exponentials (13 additions in a row, 2 +
//            2.3 d of each term, where the mean of d is at most ln 1024) 31, and its
//            reciprocal 2, which all scores share but which moves them against the
//            bias: 36
// Two such errors, rounded up; beside them the addition of the bias rounds once.
constexpr float kHalfStep = 5.9604645e-8f;
constexpr float kSoftmaxOff = 80.0f * kHalfStep, kSigmoidOff = 10.0f * kHalfStep;

__device__ __forceinline__ float quick_exp(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269502f);
}

template <int G, int V, int K>
__global__ void __launch_bounds__(256, K <= 8 ? 4 : 2) route_kernel(RouteArgs a) {
  constexpr int TOKENS = 256 / G, N = 4 * V;
  // Each wave has its tokens' part of both.
  __shared__ __attribute__((aligned(16))) uint32_t keys[TOKENS * N * G];
  // Eight tokens' rows begin on different banks.
  __shared__ __attribute__((aligned(16))) int ids[TOKENS][kRouteTop + 4];
  __shared__ int candidates[TOKENS];
  static_assert(64 / G * N * G * 4 >= N * G * 8, "a wave's keys hold one token's FP64 scores");
  const int lane = (int)threadIdx.x & 63, g = (int)threadIdx.x % G;
  const int sub = (int)threadIdx.x / G;
  const int64_t t0 = (int64_t)blockIdx.x * TOKENS + sub;
  const bool live = t0 < a.T;
  const int64_t t = live ? t0 : a.T - 1;
  const float* const row = a.logits + t * a.ld;
  const bool by_score = a.bias || (a.groups > 1 && a.group_best > 1);
  const bool whole = a.scoring == SGEMM_SCORE_SOFTMAX && (by_score || !a.renormalize);

  // The logits; -infinity: not to be chosen.
  float c[N];
  const int last = 4 * ((a.E - 1) / 4);   // where the last group of four begins
  auto row_of = [&](const float* p, f32x4 (&v)[V]) {
    if (a.E % 4 == 0) {   // without a branch for each
#pragma unroll
      for (int i = 0; i < V; ++i)
        v[i] = *reinterpret_cast<const f32x4u*>(p + min(4 * (g + i * G), last));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int col = min(4 * (g + i * G), last);
        v[i] = load_upto(p + col, a.E - col);
      }
    }
  };
  {
    f32x4 v[V];
    row_of(row, v);
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = v[i >> 2][i & 3];
  }
  if (a.E < N * G) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      c[i] = 4 * (g + (i >> 2) * G) + (i & 3) < a.E ? c[i] : -INFINITY;
  }
  float lowest = c[0];
#pragma unroll
  for (int i = 1; i < N; ++i) lowest = fminf(lowest, c[i]);
  // Rarely any of the wave's: one bit each, so that the logits need not be kept.
  const bool masked = __ballot(lowest == -INFINITY) != 0;
  static_assert(N <= 32, "a bit for each of a lane's experts");
  uint32_t never = 0u;
  if (masked) {
#pragma unroll
    for (int i = 0; i < N; ++i) never |= c[i] == -INFINITY ? 1u << i : 0u;
  }
  float top = -INFINITY, inv = 1.0f;   // of the whole softmax
  float off = kSigmoidOff;
  if (whole) {
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, c[i]);
    top = group_max<G>(top);
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float p = quick_exp(c[i] - top);   // 0 for -infinity
      sum[i & 3] += p;
      if (by_score) c[i] = p;
    }
    inv = 1.0f / group_sum<G>((sum[0] + sum[1]) + (sum[2] + sum[3]));
    off = kSoftmaxOff * inv;
  }
  uint32_t key[N];
  if (by_score) {
    f32x4 b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (a.bias) row_of(a.bias, b);
    // A score and a bias are -0 together only where the score is 0.
    auto score_key = [&](float s, int i) {
      return ordered_bits(fminf(s + b[i >> 2][i & 3], INFINITY));
    };
    if (whole) {
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = score_key(c[i] * inv, i);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        key[i] = score_key(__builtin_amdgcn_rcpf(1.0f + quick_exp(-c[i])), i);
    }
    if (masked) {
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = never >> i & 1 ? kNever : key[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = ordered(c[i]);
  }
  bool regroup = false, unsure = false;   // of the groups, of the experts
  // Groups that stay of at most half of the experts: each lane takes quads of theirs
  // alone, the first half of its keys, and the rest is not looked at again.
  constexpr int HALF = V > 1 ? V / 2 : 1;
  const bool fewer = V > 1 && a.size % 4 == 0 && 2 * a.top_groups * a.size <= N * G;
  int quad[V];
#pragma unroll
  for (int i = 0; i < V; ++i) quad[i] = g + i * G;

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
    float wide[ROUNDS];   // how far off a total may be
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const int q = r * G + g;
      total[r] = kNever;
      wide[r] = 0.0f;
      if (r * G < a.groups && q < a.groups) {
        uint32_t best = kNever, second = kNever;
        // Neighbouring groups may begin on the same bank: lanes start apart.
        if (size % 4 == 0) {
          int at = 4 * g % size;
#pragma unroll 4
          for (int i = 0; i < size; i += 4) {
            const u32x4 k = *reinterpret_cast<const u32x4*>(mine + q * size + at);
            at = at + 4 == size ? 0 : at + 4;
            const uint32_t h0 = max(k[0], k[1]), l0 = min(k[0], k[1]);
            const uint32_t h1 = max(k[2], k[3]), l1 = min(k[2], k[3]);
            const uint32_t h = max(h0, h1);
            second = max(max(second, min(best, h)), max(max(l0, l1), min(h0, h1)));
            best = max(best, h);
          }
        } else {
          int at = g % size;
          for (int i = 0; i < size; ++i) {
            const uint32_t k = mine[q * size + at];
            at = at + 1 == size ? 0 : at + 1;
            second = max(second, min(k, best));
            best = max(best, k);
          }
        }
        const bool two = a.group_best == 2 && second != kNever;
        const float x = unordered(best), y = two ? unordered(second) : 0.0f;
        total[r] = two ? ordered(x + y) : best;
        // Each score of a total is off by half of `off` and rounded at its own size, which
        // may be far larger than their sum's: at most 2 half steps of |x| + |y| with the
        // sum's own rounding, and two more for those of these bounds.
        if (fabsf(x) < INFINITY) wide[r] = off + 4.0f * kHalfStep * (fabsf(x) + fabsf(y));
      }
    }
    uint32_t* const totals = reinterpret_cast<uint32_t*>(ids[sub]);
    static_assert(kRouteTop >= SGEMM_MOE_MAX_GROUPS, "room for the groups' totals");
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
      if (r * G < a.groups) totals[r * G + g] = r * G + g < a.groups ? total[r] : 0u;
    wave_lds_fence();
    uint32_t stays = 0;
    int rank_of[ROUNDS];
    // The least that one that stays may be, the most that one that does not may be.
    float low = INFINITY, high = -INFINITY;
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      if (r * G < a.groups) {
        const int q = r * G + g;
        int rank = q < a.groups ? 0 : a.groups;
        for (int o = 0; o < a.groups; o += 4) {   // past the last one, zeros
          const u32x4 other = *reinterpret_cast<const u32x4*>(totals + o);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            rank += other[e] > total[r] || (other[e] == total[r] && o + e < q) ? 1 : 0;
        }
        rank_of[r] = rank;
        // A total past FP32, or of scores with NaN, may be anything.
        const float at = unordered(total[r]);
        const bool known = wide[r] < INFINITY;
        if (rank < a.top_groups) low = fminf(low, known ? at - wide[r] : -INFINITY);
        else if (q < a.groups) high = fmaxf(high, known ? at + wide[r] : INFINITY);
        const uint64_t bits = __ballot(rank < a.top_groups) >> (lane - g);
        stays |= (uint32_t)(bits & ((uint64_t(1) << G) - 1)) << (r * G);
      }
    }
    if (by_score && a.top_groups < a.groups) {
      butterfly<G>([&](auto s) {
        low = fminf(low, exchanged<decltype(s)::value>(low));
        high = fmaxf(high, exchanged<decltype(s)::value>(high));
      });
      regroup = high > -INFINITY && low <= high;
    }
    if (fewer) {
      wave_lds_fence();
#pragma unroll
      for (int r = 0; r < ROUNDS; ++r)
        if (r * G < a.groups && rank_of[r] < a.top_groups) ids[sub][rank_of[r]] = r * G + g;
      wave_lds_fence();
#pragma unroll
      for (int i = 0; i < HALF; ++i) {
        const int at = 4 * (g + i * G), n = group_of(a, at);   // of those that stay
        u32x4 v = {kNever, kNever, kNever, kNever};
        if (n < a.top_groups) {
          const int first = ids[sub][n] * size + at - n * size;
          quad[i] = first >> 2;
          v = *reinterpret_cast<const u32x4*>(mine + first);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) key[4 * i + e] = v[e];
      }
#pragma unroll
      for (int i = 4 * HALF; i < N; ++i) key[i] = kNever;
    } else if (size % 4 == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool gone = !(stays >> group_of(a, min(4 * (g + i * G), last)) & 1);
#pragma unroll
        for (int e = 0; e < 4; ++e) key[4 * i + e] = gone ? kNever : key[4 * i + e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = min(4 * (g + (i >> 2) * G) + (i & 3), a.E - 1);
        key[i] = stays >> group_of(a, e) & 1 ? key[i] : kNever;
      }
    }
  }

  // This lane's best K, then all lanes'.
  double best[K];
#pragma unroll
  for (int i0 = 0; i0 < N; i0 += K) {
    if (i0 >= 4 * HALF && fewer) continue;
    double v[K];
#pragma unroll
    for (int j = 0; j < K; ++j)
      v[j] = i0 + j < N ? packed(key[i0 + j < N ? i0 + j : 0],
                                 4 * quad[(i0 + j < N ? i0 + j : 0) >> 2] + ((i0 + j) & 3))
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
  constexpr int J = (K + G - 1) / G;   // lane g has choices g, g + G ..
#pragma unroll
  for (int r = 0; r < J; ++r) {
    double mine = best[r * G];
#pragma unroll
    for (int j = 1; j < G && r * G + j < K; ++j) mine = g == j ? best[r * G + j] : mine;
    if (r * G + g < a.top) ids[sub][r * G + g] = packed_expert(mine);
  }

  if (by_score) {
    // How far below a score another may be and yet be the larger one, for the largest
    // of the list: both errors, and each one's rounding (a little more, as the lower
    // one's size may exceed the other's by as much).
    float far = 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const uint32_t k = packed_key(best[j]);
      far = fmaxf(far, k > kNever ? fabsf(unordered(k)) : 0.0f);
    }
    const float reach = 1.01f * (off + 4.0f * kHalfStep * far);
    uint32_t from = 0u, chosen = 0u;   // of the last one chosen
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const uint32_t k = packed_key(best[j]), down_to = ordered(unordered(k) - reach);
      if (j + 1 < K && j + 1 < a.top) {
        const uint32_t after = packed_key(best[j + 1 < K ? j + 1 : 0]);
        unsure |= (after > kNever) & (after >= down_to);
      }
      if (j == a.top - 1) {
        chosen = k;
        from = down_to;
      }
    }
    // No other may be within reach of the last one.
    int close = 0;
#pragma unroll
    for (int i = 0; i < 4 * HALF; ++i) close += key[i] >= from ? 1 : 0;
    if (!fewer) {
#pragma unroll
      for (int i = 4 * HALF; i < N; ++i) close += key[i] >= from ? 1 : 0;
    }
    close = group_sum<G>(close);
    unsure |= (chosen > kNever) & (close > a.top);
    // A token's lanes agree on both.
    if (__ballot((unsure || regroup) && live) != 0) {
      constexpr int MOST = N * G < 64 ? N * G : 64;
      const int first = sub - lane / G;   // the wave's first token
      int* const list = reinterpret_cast<int*>(keys + sub * (N * G));
      if (g == 0) candidates[sub] = 0;
      wave_lds_fence();
      if (unsure && !regroup) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (key[i] >= from && key[i] > kNever) {
            const int slot = atomicAdd(&candidates[sub], 1);
            if (slot < MOST) list[slot] = 4 * quad[i >> 2] + (i & 3);
          }
        }
      }
      wave_lds_fence();
      const bool whole_choice = regroup || candidates[sub] > MOST;
      constexpr int Q = (N * G + 63) / 64;
      auto each = [&](bool mine, auto f) {
        for (uint64_t left = __ballot(mine && live); left != 0;) {
          const int of = (__ffsll((unsigned long long)left) - 1) / G;   // of the wave's tokens
          f(first + of, (int64_t)blockIdx.x * TOKENS + first + of);
          left &= ~(((uint64_t(1) << G) - 1) << (of * G));
        }
      };
      each(unsure && !whole_choice, [&](int at, int64_t token) {
        reorder<Q>(a, token, reinterpret_cast<const int*>(keys + at * (N * G)), candidates[at],
                   ids[at]);
      });
      wave_lds_fence();
      // These need the lists' room.
      each(whole_choice, [&](int at, int64_t token) {
        refine<Q>(a, token, reinterpret_cast<double*>(keys + first * (N * G)), ids[at]);
      });
    }
  }
  wave_lds_fence();

  // Weights.
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
