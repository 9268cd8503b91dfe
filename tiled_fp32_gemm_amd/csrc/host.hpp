// host.hpp -- host-side helpers shared by the entry points: operand spans and
// overlaps, grid limits, and the time model the planners choose tiles with.
#pragma once

#include <stdint.h>

#include "common.hpp"

namespace sg {
namespace host {

// The kernels address each operand from the corner of their own tile with
// 32-bit byte offsets below 2^31 (kOob = 2^31 marks an element outside the
// matrix), so what is bounded is one tile's span, not an operand's size.
constexpr int64_t kMaxSpanBytes = sg::kRsrcMax;
// Tile origins and sizes are 32-bit ints in the kernels.
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;
// Bytes spanned by a rows x cols row-major operand with leading dimension ld
// (0 when empty); -1 when the span does not fit in int64.
inline int64_t span_bytes(int64_t rows, int64_t cols, int64_t ld) {
  if (rows == 0 || cols == 0) return 0;
  const int64_t lim = INT64_MAX / 4;
  if (rows - 1 > (lim - cols) / ld) return -1;
  return ((rows - 1) * ld + cols) * 4;
}

inline bool overlaps(const void* p, int64_t pb, const void* q, int64_t qb) {
  if (pb == 0 || qb == 0) return false;
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + (uintptr_t)qb && b < a + (uintptr_t)pb;
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// True when rows x width floats with leading dimension ld (the first row
// starting at offset 0) end below kMaxSpanBytes: ((rows - 1) ld + width) 4
// bytes, formed without overflow.
inline bool span_fits(int64_t rows, int64_t width, int64_t ld) {
  if (rows <= 0 || width <= 0) return true;
  const int64_t lim = kMaxSpanBytes / 4;  // floats
  if (width >= lim) return false;
  if (rows == 1) return true;
  if (ld > (lim - 1 - width) / (rows - 1)) return false;
  return (rows - 1) * ld + width < lim;
}

// The grid's work-items, workgroups x threads, must fit in 32 bits.
inline bool grid_fits(int64_t workgroups, int threads) {
  return workgroups >= 0 && workgroups < ((int64_t(1) << 32) / threads);
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kCUs = 256;                      // MI355X compute units
constexpr double kPeakPerCU = 157.3e12 / kCUs;  // FP32 matrix flop/s per CU
constexpr double kSaturate = 1.28;   // waves per SIMD that keep the pipes busy
constexpr double kSlabFloor = 0.61e-6;  // s: a slab's wait for its loads
constexpr double kRoundCost = 4.4e-6;   // s: fill and drain of one round
constexpr double kWriteBW = 4.52e12;    // B/s: C stores of a final round
constexpr double kReduceFixed = 3.0e-6;  // s: the second launch of a split product
constexpr double kReduceBW = 5.0e12;     // B/s, a device copy's rate


// What the time model needs to know of a tile variant.
struct TileCost {
  int tile_m, tile_n, tile_k, threads;
  double eff;   // fraction of a CU's FP32 matrix peak with its pipes busy
  int occ;      // workgroups a CU holds at once
  double slab_floor = kSlabFloor;   // s a slab takes however little it computes
  double saturate = kSaturate;      // waves per SIMD that keep the pipes busy
  double round_more = 0.0;          // s a round takes beside kRoundCost
};

// Estimated seconds of a tile variant on an M x N x K product.  Workgroups are
// spread evenly over the CUs, so the busiest CU computes n = ceil(tiles /
// CUs) tiles (charging partial-tile padding and the idle CUs of the last
// round, i.e. wave quantisation), in rounds of up to occ resident ones.  In a
// round of r tiles every slab takes the longer of its compute (r tiles'
// flops at eff of the CU's peak, in proportion below kSaturate waves per
// SIMD) and the latency of its loads; each round adds a fixed cost; and the
// C tiles of the final round, which all CUs store at once, are charged at
// the chip's write bandwidth.
inline double estimate_grid(const TileCost& v, int64_t tiles, int64_t K) {
  const int64_t n = cdiv(tiles, kCUs);
  const int64_t slabs = K > v.tile_k ? cdiv(K, v.tile_k) : 1;
  const double waves = v.threads / 64.0;
  const double slab_flops = 2.0 * v.tile_m * v.tile_n * v.tile_k;
  auto round = [&](int64_t r) {
    const double simd = r * waves / 4.0;
    const double busy = simd >= v.saturate ? 1.0 : simd / v.saturate;
    const double compute = r * slab_flops / (kPeakPerCU * v.eff * busy);
    return (double)slabs * (compute > v.slab_floor ? compute : v.slab_floor) + kRoundCost +
           v.round_more;
  };
  const int64_t full = n / v.occ, rest = n % v.occ;
  double t = (double)full * round(v.occ) + (rest > 0 ? round(rest) : 0.0);
  const int64_t last = rest > 0 ? rest : v.occ;
  const int64_t cus = tiles < kCUs ? tiles : kCUs;
  t += (double)last * cus * v.tile_m * v.tile_n * 4.0 / kWriteBW;
  return t;
}

}  // namespace host
}  // namespace sg
