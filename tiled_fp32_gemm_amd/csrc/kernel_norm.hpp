// kernel_norm.hpp -- layer norm over rows, and its gradients.
//
// A row lies in the registers of L lanes, V groups of four columns each: it is
// read once, its mean is summed, then the squares of what is left of the mean
// (the sum of squares less the squared mean would cancel where the mean is
// large), and the result is written.  The lanes take row after row and load the
// next one before they sum the present one; weight and bias stay in their
// registers.  Rows wider than any such variant are read again for each step by a
// workgroup of 1024 (norm_wide_*).
//
// The gradients need dy and x once as well.  A workgroup adds dy xh and dy of
// its rows column by column in registers, puts its waves' sums together in LDS
// and leaves one row of 2 N sums in the workspace; norm_sum_kernel adds those
// rows in a fixed order.  There are workgroups enough that a lane adds no more than
// kNormRun rows: the rounding errors grow with n / 256 + 256 rather than n.
//
// Bound by HBM: 8 bytes an element forward, 12 backward (16 with a residual).
// Measured on MI355X (averages): 32768 x 4096 forward 201 us (5.3 TB/s), 4000 x 16384 103
// (5.1), 16 x 1024 3.5; the gradients of 32768 x 1024 with a residual 84 + 5 us (6.0 TB/s), of
// 4000 x 8192 70 + 8 (5.0), of 1000 x 777 6.3 + 3.8.
//
// A workgroup of 1024 has 128 registers a lane.  Forward, four groups of four columns
// take 64 of them (a row, the next one, weight, bias): up to 16384 columns.  Backward, two
// take 64 (dy, x and the next ones, weight, residual and both sums), four would take
// all: up to 8192.  The wide kernels past that read a row from the caches for their
// second and third step: 4000 x 20000 forward 175 us (3.7 TB/s of what has to move);
// backward 4000 x 12288  139 + 92 + 9, 4000 x 16384  187 + 114 + 9 (2.5).
#pragma once

#include "lanes.hpp"
#include "rows.hpp"

namespace sg {

struct NormArgs {
  const float* X;
  const float* weight;   // null: 1
  const float* bias;     // null: 0
  float* Y;
  float* mean;           // null: not wanted
  float* rstd;
  int64_t ldx, ldy, M;
  int N;
  float eps;
};

// Four columns from an f32x4, zeros where there are none.
__device__ __forceinline__ f32x4 first_of(f32x4 v, int left) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = e < left ? v[e] : 0.0f;
  return v;
}

__device__ __forceinline__ float sum_of(f32x4 v) { return (v[0] + v[1]) + (v[2] + v[3]); }

template <int L>
constexpr int kNormThreads = L > 64 ? L : 256;

template <int L, int V>
__global__ void __launch_bounds__(kNormThreads<L>) norm_kernel(NormArgs a) {
  constexpr int R = kNormThreads<L> / L;   // rows at a time
  __shared__ float part[2][L > 64 ? L / 64 : 1];
  const int lane = (int)threadIdx.x % L;
  const float n = (float)a.N;
  int64_t row = (int64_t)blockIdx.x * R + (int)threadIdx.x / L;
  const int64_t step = (int64_t)gridDim.x * R;
  if (row >= a.M) return;   // whole groups of L lanes
  f32x4 x[V], w[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = 4 * (lane + i * L), left = a.N - col;
    w[i] = {1.0f, 1.0f, 1.0f, 1.0f};
    x[i] = b[i] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (left > 0) {
      x[i] = load_upto(a.X + row * a.ldx + col, left);
      if (a.weight) w[i] = load_upto(a.weight + col, left);
      if (a.bias) b[i] = load_upto(a.bias + col, left);
    }
  }
  while (true) {
    const int64_t next = row + step;
    f32x4 ahead[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = 4 * (lane + i * L), left = a.N - col;
      ahead[i] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (next < a.M && left > 0) ahead[i] = load_upto(a.X + next * a.ldx + col, left);
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) s[0] += sum_of(x[i]);
    row_sums<L>(s, part[0]);
    const float mean = s[0] / n;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = first_of(x[i] - mean, a.N - 4 * (lane + i * L));
      s[0] += sum_of(x[i] * x[i]);
    }
    row_sums<L>(s, part[1]);
    const float rstd = 1.0f / sqrtf(s[0] / n + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = 4 * (lane + i * L), left = a.N - col;
      if (left > 0) store_upto(a.Y + row * a.ldy + col, left, x[i] * rstd * w[i] + b[i]);
    }
    if (lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    if (next >= a.M) return;
    row = next;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = ahead[i];
  }
}

// Rows of any width, one a workgroup.
__global__ void __launch_bounds__(1024) norm_wide_kernel(NormArgs a) {
  __shared__ float part[2][16];
  const int64_t row = blockIdx.x;
  const float* const x = a.X + row * a.ldx;
  const float n = (float)a.N;
  auto sum = [&](float mean, bool squares, float* room) {
    f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t col = 4 * (int)threadIdx.x; col < a.N; col += 4096) {
      const int left = (int)(a.N - col);
      const f32x4 d = first_of(load_upto(x + col, left) - mean, left);
      t += squares ? d * d : d;
    }
    float s[1] = {sum_of(t)};
    row_sums<1024>(s, room);
    return s[0] / n;
  };
  const float mean = sum(0.0f, false, part[0]);
  const float rstd = 1.0f / sqrtf(sum(mean, true, part[1]) + a.eps);
  for (int64_t col = 4 * (int)threadIdx.x; col < a.N; col += 4096) {
    const int left = (int)(a.N - col);
    f32x4 y = (load_upto(x + col, left) - mean) * rstd;
    if (a.weight) y *= load_upto(a.weight + col, left);
    if (a.bias) y += load_upto(a.bias + col, left);
    store_upto(a.Y + row * a.ldy + col, left, y);
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

struct NormBackwardArgs {
  const float* dY;
  const float* X;
  const float* mean;
  const float* rstd;
  const float* weight;     // null: 1
  const float* residual;   // null: none
  float* dX;               // null: only the sums
  float* W;                // [span][2 N]: dweight's and dbias' sums; null: not wanted
  float* dweight;
  float* dbias;
  int64_t lddy, ldx, ldr, lddx, M;
  int N, spans;
};

constexpr int kNormRun = 256;

template <int L, int V>
__global__ void __launch_bounds__(kNormThreads<L>) norm_backward_kernel(NormBackwardArgs a) {
  constexpr int R = kNormThreads<L> / L, ROW = 4 * L * V;
  __shared__ float part[2][L > 64 ? L / 32 : 1];
  __shared__ __attribute__((aligned(16))) float sums[R > 1 ? R * ROW : 4];
  const int lane = (int)threadIdx.x % L, sub = (int)threadIdx.x / L;
  const float inv = 1.0f / (float)a.N;
  int64_t row = (int64_t)blockIdx.x * R + sub;
  const int64_t step = (int64_t)gridDim.x * R;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 dy[V], x[V], w[V], dw[V], db[V];
  float mean = 0.0f, rstd = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = 4 * (lane + i * L), left = a.N - col;
    w[i] = {1.0f, 1.0f, 1.0f, 1.0f};
    dy[i] = x[i] = dw[i] = db[i] = zero;
    if (left > 0) {
      if (row < a.M) {
        dy[i] = load_upto_once(a.dY + row * a.lddy + col, left);
        x[i] = load_upto_once(a.X + row * a.ldx + col, left);
      }
      if (a.weight) w[i] = load_upto(a.weight + col, left);
    }
  }
  if (row < a.M) {
    mean = a.mean[row];
    rstd = a.rstd[row];
  }
  int odd = 0;   // which half of `part`
  while (row < a.M) {
    const int64_t next = row + step;
    f32x4 dy_ahead[V], x_ahead[V], res[V];
    float mean_ahead = 0.0f, rstd_ahead = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = 4 * (lane + i * L), left = a.N - col;
      dy_ahead[i] = x_ahead[i] = res[i] = zero;
      if (left > 0 && a.dX && a.residual)
        res[i] = load_upto_once(a.residual + row * a.ldr + col, left);
      if (left > 0 && next < a.M) {
        dy_ahead[i] = load_upto_once(a.dY + next * a.lddy + col, left);
        x_ahead[i] = load_upto_once(a.X + next * a.ldx + col, left);
      }
    }
    if (next < a.M) {
      mean_ahead = a.mean[next];
      rstd_ahead = a.rstd[next];
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = first_of((x[i] - mean) * rstd, a.N - 4 * (lane + i * L));   // xh
      dw[i] += dy[i] * x[i];
      db[i] += dy[i];
      dy[i] *= w[i];
      s[0] += sum_of(dy[i]);
      s[1] += sum_of(dy[i] * x[i]);
    }
    if (a.dX) {
      row_sums<L>(s, part[odd]);
      odd ^= 1;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int col = 4 * (lane + i * L), left = a.N - col;
        const f32x4 d = (dy[i] - s[0] * inv - x[i] * (s[1] * inv)) * rstd + res[i];
        if (left > 0) store_upto(a.dX + row * a.lddx + col, left, d);
      }
    }
    row = next;
    mean = mean_ahead;
    rstd = rstd_ahead;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dy[i] = dy_ahead[i];
      x[i] = x_ahead[i];
    }
  }
  if (!a.W) return;
  // The rows side by side, then this workgroup's row of the workspace.
  float* const out = a.W + (int64_t)blockIdx.x * 2 * a.N;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if constexpr (R > 1) {
      f32x4* const mine = reinterpret_cast<f32x4*>(sums) + sub * (ROW / 4) + lane;
      if (k > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) mine[i * L] = k == 0 ? dw[i] : db[i];
      __syncthreads();
      for (int q = (int)threadIdx.x; q < ROW / 4; q += kNormThreads<L>) {
        const int left = a.N - 4 * q;
        if (left <= 0) break;
        f32x4 t = reinterpret_cast<f32x4*>(sums)[q];
#pragma unroll
        for (int r = 1; r < R; ++r) t += reinterpret_cast<f32x4*>(sums)[r * (ROW / 4) + q];
        store_upto(out + (int64_t)k * a.N + 4 * q, left, t);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int col = 4 * (lane + i * L), left = a.N - col;
        if (left > 0) store_upto(out + (int64_t)k * a.N + col, left, k == 0 ? dw[i] : db[i]);
      }
    }
  }
}

// Rows of any width: dX, one row a workgroup.
__global__ void __launch_bounds__(1024) norm_wide_backward_kernel(NormBackwardArgs a) {
  __shared__ float part[32];
  const int64_t row = blockIdx.x;
  const float* const dy = a.dY + row * a.lddy;
  const float* const x = a.X + row * a.ldx;
  const float mean = a.mean[row], rstd = a.rstd[row], inv = 1.0f / (float)a.N;
  auto g_and_xh = [&](int64_t col, int left, f32x4& g, f32x4& xh) {
    g = load_upto(dy + col, left);
    if (a.weight) g *= load_upto(a.weight + col, left);
    xh = first_of((load_upto(x + col, left) - mean) * rstd, left);
  };
  f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f}, u = t, g, xh;
  for (int64_t col = 4 * (int)threadIdx.x; col < a.N; col += 4096) {
    g_and_xh(col, (int)(a.N - col), g, xh);
    t += g;
    u += g * xh;
  }
  float s[2] = {sum_of(t), sum_of(u)};
  row_sums<1024>(s, part);
  for (int64_t col = 4 * (int)threadIdx.x; col < a.N; col += 4096) {
    const int left = (int)(a.N - col);
    g_and_xh(col, left, g, xh);
    f32x4 d = (g - s[0] * inv - xh * (s[1] * inv)) * rstd;
    if (a.residual) d += load_upto(a.residual + row * a.ldr + col, left);
    store_upto(a.dX + row * a.lddx + col, left, d);
  }
}

// Rows of any width: a span's sums, 1024 columns a workgroup.
constexpr int kNormWideCols = 1024;

__global__ void __launch_bounds__(256) norm_wide_sums_kernel(NormBackwardArgs a) {
  const int blocks = (a.N + kNormWideCols - 1) / kNormWideCols;
  const int span = (int)(blockIdx.x / (unsigned)blocks);
  const int64_t col = (int64_t)(blockIdx.x % (unsigned)blocks) * kNormWideCols +
                      4 * (int)threadIdx.x;
  const int left = (int)min((int64_t)4, a.N - col);
  if (left <= 0) return;
  f32x4 dw = {0.0f, 0.0f, 0.0f, 0.0f}, db = dw;
#pragma unroll 4
  for (int64_t row = span; row < a.M; row += a.spans) {
    const f32x4 dy = load_upto(a.dY + row * a.lddy + col, left);
    dw += dy * ((load_upto(a.X + row * a.ldx + col, left) - a.mean[row]) * a.rstd[row]);
    db += dy;
  }
  float* const out = a.W + (int64_t)span * 2 * a.N + col;
  store_upto(out, left, dw);
  store_upto(out + a.N, left, db);
}

// dweight and dbias: the spans' rows added, 16 of the 2 N columns a workgroup.
// Span s is in part s mod 64; the parts, each added in order, meet by halves.
constexpr int kNormSumCols = 16;

__global__ void __launch_bounds__(1024) norm_sum_kernel(NormBackwardArgs a) {
  constexpr int PARTS = 1024 / kNormSumCols;
  __shared__ float part[1024];
  const int tid = (int)threadIdx.x;
  const int64_t wide = 2 * (int64_t)a.N;
  const int64_t col = (int64_t)blockIdx.x * kNormSumCols + tid % kNormSumCols;
  float sum = 0.0f;
  if (col < wide) {
    const float* p = a.W + col;
#pragma unroll 8
    for (int s = tid / kNormSumCols; s < a.spans; s += PARTS) sum += p[s * wide];
  }
  part[tid] = sum;
  for (int half = 512; half >= kNormSumCols; half /= 2) {
    __syncthreads();
    if (tid < half) part[tid] += part[tid + half];
  }
  if (tid >= kNormSumCols || col >= wide) return;
  float* const out = col < a.N ? a.dweight : a.dbias;
  if (out) out[col < a.N ? col : col - a.N] = part[tid];
}

}  // namespace sg
