// kernel_moe.hpp -- expert routing: the sort of the choices, and the rows'
// moves there and back.
//
// The sort is a stable counting sort.  Every workgroup takes one contiguous
// chunk of the choices, every wave a contiguous part of the chunk, 64 choices
// at a time: lanes with the same expert find each other by one ballot per bit
// of the expert's number, a lane's rank is the count of equal lanes before
// it, and the first of them moves the wave's counter of that expert on.  All
// counts are sums of whole numbers, so the result does not depend on timing.
// A sort of one chunk is one launch.  With more chunks a first launch counts
// each chunk's experts; the second adds up the counts of the chunks before
// its own.  Bound by latency: on MI355X 4.6 us for 32 choices, 4.6 + 9.0 us for
// 131072 choices of 64 experts.
//
// The moves read each row once and write each row once, and are bound by HBM.
// Rows are addressed with 64-bit offsets, 16 bytes a lane at any 4-byte
// alignment.  32768 tokens by four rows of 1024 floats (671 MB each way): there
// 122 us (5.5 TB/s), back 105 us (6.4 TB/s); plain instead of nontemporal
// accesses took 103 and 157 us.  The gradients of 8191 x 2 rows of 777 floats
// (127 MB): 27 us (4.7 TB/s).
#pragma once

#include "../../include/sgemm_moe.h"
#include "rows.hpp"

namespace sg {

constexpr int kMaxExperts = SGEMM_MOE_MAX_EXPERTS;

struct SortArgs {
  const void* experts;
  int32_t* offsets;
  int32_t* order;
  int32_t* place;
  int32_t* counts;   // [chunk][E]
  int n, E, chunk, chunks;
  int bits;          // of E - 1
};

template <typename Id>
__device__ __forceinline__ int expert_of(const void* experts, int i, int E) {
  const Id id = static_cast<const Id*>(experts)[i];
  return id >= 0 && id < (Id)E ? (int)id : -1;
}

template <typename Id>
__global__ void __launch_bounds__(256) moe_count_kernel(SortArgs a) {
  __shared__ int hist[kMaxExperts];
  for (int e = (int)threadIdx.x; e < a.E; e += 256) hist[e] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * a.chunk;
  const int last = (int)min(first + a.chunk, (int64_t)a.n);
  for (int64_t i = first + threadIdx.x; i < last; i += 256) {
    const int e = expert_of<Id>(a.experts, (int)i, a.E);
    if (e >= 0) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = (int)threadIdx.x; e < a.E; e += 256)
    a.counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

template <typename Id, int WAVES>
__global__ void __launch_bounds__(64 * WAVES) moe_sort_kernel(SortArgs a) {
  constexpr int NT = 64 * WAVES;
  __shared__ int next[WAVES][kMaxExperts];   // each wave's count, then its next row
  __shared__ int total[kMaxExperts];         // of all chunks, then the first row
  __shared__ int before[kMaxExperts];        // of the chunks before this one
  __shared__ int kept;
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = (int)blockIdx.x;
  for (int e = tid; e < a.E; e += NT) {
    total[e] = before[e] = 0;
    for (int w = 0; w < WAVES; ++w) next[w][e] = 0;
  }
  __syncthreads();
  const int64_t first = (int64_t)b * a.chunk;
  const int last = (int)min(first + a.chunk, (int64_t)a.n);
  const int per = ((a.chunk + WAVES - 1) / WAVES + 63) / 64 * 64;   // a wave's part
  const int64_t w0 = first + (int64_t)wave * per;
  const int64_t w1 = min(w0 + per, (int64_t)last);
#pragma unroll 4
  for (int64_t i = w0 + lane; i < w1; i += 64) {
    const int e = expert_of<Id>(a.experts, (int)i, a.E);
    if (e >= 0) atomicAdd(&next[wave][e], 1);
  }
  __syncthreads();
  if (a.chunks > 1) {   // all chunks' counts, and those of the chunks before
    const int n = a.chunks * a.E, mine = b * a.E, skip = NT % a.E;
    int e = tid % a.E;
    constexpr int U = 16;   // counts in flight
    for (int i0 = tid; i0 < n; i0 += U * NT) {
      int v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = i0 + u * NT < n ? a.counts[i0 + u * NT] : 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v[u] != 0) {
          atomicAdd(&total[e], v[u]);
          if (i0 + u * NT < mine) atomicAdd(&before[e], v[u]);
        }
        e += skip;
        if (e >= a.E) e -= a.E;
      }
    }
    __syncthreads();
  }
  // Each wave's count becomes the rows of its expert before it.
  for (int e = tid; e < a.E; e += NT) {
    int row = before[e];
    for (int w = 0; w < WAVES; ++w) {
      const int v = next[w][e];
      next[w][e] = row;
      row += v;
    }
    if (a.chunks == 1) total[e] = row;
  }
  __syncthreads();
  if (wave == 0) {   // exclusive scan of the totals
    int run = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + lane;
      const int v = e < a.E ? total[e] : 0;
      int s = v;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(s, d);
        if (lane >= d) s += o;
      }
      if (e < a.E) total[e] = run + s - v;
      run += __shfl(s, 63);
    }
    if (lane == 0) kept = run;
  }
  __syncthreads();
  if (b == 0) {
    for (int e = tid; e < a.E; e += NT) a.offsets[e] = total[e];
    if (tid == 0) a.offsets[a.E] = kept;
  }
  for (int64_t r = first + tid; r < last; r += NT)   // this chunk's share of the rows
    if (r >= kept) a.order[r] = -1;
  int ahead = w0 + lane < w1 ? expert_of<Id>(a.experts, (int)(w0 + lane), a.E) : -1;
  for (int64_t i0 = w0; i0 < w1; i0 += 64) {
    const int64_t i = i0 + lane;
    const bool in = i < w1;
    const int e = ahead;
    ahead = i + 64 < w1 ? expert_of<Id>(a.experts, (int)i + 64, a.E) : -1;
    uint64_t same = __ballot(e >= 0);
    for (int k = 0; k < a.bits; ++k) {
      const bool bit = (e >> k) & 1;
      const uint64_t set = __ballot(bit);
      same &= bit ? set : ~set;
    }
    int row = 0;
    const int leader = e >= 0 ? __ffsll((unsigned long long)same) - 1 : lane;
    if (e >= 0 && lane == leader) row = atomicAdd(&next[wave][e], __popcll(same));
    row = __shfl(row, leader);
    if (e >= 0) {
      row += total[e] + __popcll(same & ((uint64_t(1) << lane) - 1));
      a.order[row] = (int)i;
      a.place[i] = row;
    } else if (in) {
      a.place[i] = -1;
    }
  }
}

struct MoveArgs {
  const float* in;        // permute: X;  unpermute: Yp;  backward: Yp
  const float* grad;      // backward: dY
  float* out;             // permute: Xp; unpermute: Y;   backward: dYp
  float* dweights;
  const float* weights;
  const int32_t* place;
  int64_t ld_in, ld_grad, ld_out;
  int64_t T;
  int top, H, rows;       // rows = T top
};

// The token and the first of the four columns of this thread: the rows' 16-byte
// groups are numbered through, so that every lane has one whatever H is.
__device__ __forceinline__ bool move_place(const MoveArgs& a, int64_t& t, int& col) {
  const int groups = (a.H + 3) / 4;
  const int64_t first = (int64_t)blockIdx.x * 256;
  const int64_t t0 = first / groups;
  const unsigned in = (unsigned)(first - t0 * groups) + threadIdx.x;
  const unsigned down = in / (unsigned)groups;
  t = t0 + down;
  col = 4 * (int)(in - down * (unsigned)groups);
  return t < a.T;
}

__global__ void __launch_bounds__(256) moe_permute_kernel(MoveArgs a) {
  int64_t t;
  int col;
  if (!move_place(a, t, col)) return;
  const int n = a.H - col;
  const f32x4 v = load_upto_once(a.in + t * a.ld_in + col, n);
  for (int j = 0; j < a.top; ++j) {
    const int p = a.place[t * a.top + j];
    if (p >= 0 && p < a.rows) store_upto_once(a.out + p * a.ld_out + col, n, v);
  }
}

__global__ void __launch_bounds__(256) moe_unpermute_kernel(MoveArgs a) {
  int64_t t;
  int col;
  if (!move_place(a, t, col)) return;
  const int n = a.H - col;
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = 4;
  for (int j0 = 0; j0 < a.top; j0 += U) {
    f32x4 v[U];
    float w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      w[u] = 0.0f;
      v[u] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (j0 + u < a.top) {
        const int64_t c = t * a.top + j0 + u;
        const int p = a.place[c];
        if (p >= 0 && p < a.rows) {
          w[u] = a.weights ? a.weights[c] : 1.0f;
          v[u] = load_upto_once(a.in + p * a.ld_in + col, n);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = fmaf(w[u], v[u][e], sum[e]);
  }
  store_upto_once(a.out + t * a.ld_out + col, n, sum);
}

// G lanes per choice.
template <int G>
__global__ void __launch_bounds__(256) moe_unpermute_backward_kernel(MoveArgs a) {
  const int64_t c = (int64_t)blockIdx.x * (256 / G) + (int)threadIdx.x / G;
  const int lane = (int)threadIdx.x % G;
  if (c >= a.rows) return;   // whole groups of G lanes
  const int p = a.place[c];
  if (p < 0 || p >= a.rows) {
    if (a.dweights && lane == 0) a.dweights[c] = 0.0f;
    return;
  }
  const float w = a.weights ? a.weights[c] : 1.0f;
  const float* g = a.grad + (c / a.top) * a.ld_grad;
  const float* y = a.in + p * a.ld_in;
  float* o = a.out + p * a.ld_out;
  f32x4 dot = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = 4;   // groups in flight
  for (int c0 = 4 * lane; c0 < a.H; c0 += U * 4 * G) {
    f32x4 d[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int col = c0 + u * 4 * G, n = a.H - col;
      d[u] = v[u] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (n > 0) {
        d[u] = load_upto(g + col, n);
        if (a.dweights) v[u] = load_upto_once(y + col, n);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int col = c0 + u * 4 * G, n = a.H - col;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dot[e] = fmaf(d[u][e], v[u][e], dot[e]);
        d[u][e] *= w;
      }
      if (a.out && n > 0) store_upto_once(o + col, n, d[u]);
    }
  }
  if (!a.dweights) return;
  float s = (dot[0] + dot[1]) + (dot[2] + dot[3]);
#pragma unroll
  for (int d = G / 2; d > 0; d >>= 1) s += __shfl_xor(s, d, G);
  if (lane == 0) a.dweights[c] = s;
}

}  // namespace sg
