// xent.hip -- the C ABI of include/sgemm_xent.h: argument checks, the plan and its
// launches.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <string.h>

#include "../../include/sgemm_linear.h"
#include "../../include/sgemm_moe.h"
#include "../../include/sgemm_xent.h"
#include "kernel_xent.hpp"
#include "kernel_xent_few.hpp"
#include "product_planes.hpp"

namespace {

using namespace sg::host;
using sg::Targets;
using sg::XentFewArgs;
using sg::XentFewSumArgs;
using sg::XentLossArgs;
using sg::XentPlaceArgs;
using sg::XentPlanesArgs;
using sg::XentProductArgs;
using sg::XentRows;
using sg::XentVariant;

struct Span {
  const void* p;
  int64_t bytes;   // 0: not touched; -1: beyond int64
};

bool overlaps(const Span& a, const Span& b) {
  return sg::host::overlaps(a.p, a.bytes, b.p, b.bytes);
}

bool bad(const Span& s) { return s.bytes != 0 && (s.p == nullptr || ((uintptr_t)s.p & 3u)); }

int64_t at_least_one(int64_t n) { return n > 1 ? n : 1; }
int64_t round_up(int64_t n, int64_t to) { return cdiv(n, to) * to; }

// A leading dimension only matters past the first row.
int64_t leading(int64_t rows, int64_t width, int64_t ld) {
  return rows > 1 ? ld : at_least_one(width);
}

bool sizes_ok(int64_t T, int64_t V, int64_t H) {
  return T >= 0 && V >= 0 && H >= 0 && T <= kMaxDim && V <= SGEMM_XENT_MAX_LD &&
         H <= SGEMM_XENT_MAX_LD;
}

// The tile with the least estimated time for T x V over H; null: no grid holds it.
const XentVariant* choose(bool trans_b, int64_t T, int64_t V, int64_t H) {
  const XentVariant* table = trans_b ? sg::xent_variants_ff() : sg::xent_variants_fs();
  const XentVariant* best = nullptr;
  double t_best = 0.0;
  for (int i = 0; i < sg::kXentVariants; ++i) {
    const TileCost& c = table[i].cost;
    const int64_t tiles = cdiv(T, c.tile_m) * cdiv(V, c.tile_n);
    if (!grid_fits(tiles, c.threads)) continue;
    const double t = estimate_grid(c, tiles, H);
    if (best == nullptr || t < t_best * 0.995) {
      best = &table[i];
      t_best = t;
    }
  }
  return best;
}

// A workspace handed out front to back, each part on 16 bytes of it.
struct Room {
  char* p;
  int64_t used;
  template <class T>
  T* take(int64_t n) {
    T* at = p ? reinterpret_cast<T*>(p + used) : nullptr;
    used += round_up(n * (int64_t)sizeof(T), 16);
    return at;
  }
};

XentRows take_rows(Room& room, int64_t T, int64_t H, bool backward) {
  XentRows r = {};
  r.offsets = room.take<int32_t>(2);
  r.place = room.take<int32_t>(T);
  if (backward) r.row = room.take<sg::XentRow>(T);
  else r.target = room.take<int32_t>(T);
  r.X = room.take<float>(T * H);
  return r;
}

// Copying the rows together takes some 10 us and their traffic, a hundredth of a
// product that takes this long, and saves the products of the rows left out.
constexpr double kGatherSeconds = 200e-6;

// The copies' grid, four values a thread.
bool rows_fit(int64_t T, int64_t H) { return grid_fits(cdiv(T * cdiv(H, 4), 256), 256); }

constexpr int64_t kLossRowsFrom = 1024;   // tokens

// How many planes (product_planes.hpp) T x V over H is best left in; 0: rather tiles
// that end in a row's statistics or gradient.  Planes win where K has to be split to
// fill the chip, and where up to eight rows over a large B need no tiles.  Measured
// (forward us, tiles / planes; T, H, V, B stored V x H or H x V):
//      split        19, 2894, 3306 H x V 43 / 22, 3, 2647, 111 H x V 28 / 18,
//                   300, 4096, 500 V x H 40 / 24, 1000, 4096, 300 V x H 41 / 34
//      by rows      1, 1024, 32768 V x H 39 / 31, 8 rows 38 / 37, H x V 34 / 32,
//                   1, 4096, 65536 V x H 213 / 174, 1, 512, 1000 V x H 12.6 / 14.9
//      16 rows (B twice)  1024, 32768 V x H 38 / 43;  one plane by tiles  200, 1024,
//                   2000 V x H 18 / 20
constexpr int64_t kPlanesOne = int64_t(16) << 20, kPlanesAll = int64_t(64) << 20;   // bytes

int choose_planes(const XentVariant* v, bool grouped, bool trans_b, int64_t T, int64_t V,
                  int64_t H) {
  const int64_t one = 4 * T * V;
  if (v == nullptr || one == 0 || H == 0 || one > kPlanesOne) return 0;
  const PlanesPlan plan = plan_planes(grouped, trans_b, T, V, H, kPlanesAll);
  if (!plan.possible || (plan.count == 1 && !plan.rows)) return 0;
  const int64_t tiles = cdiv(T, v->cost.tile_m) * cdiv(V, v->cost.tile_n);
  const double b = 4.0 * V * H, by_tiles = estimate_grid(v->cost, tiles, H);
  // A split's time has a second pass already; after rows it is a launch more.
  if (plan.count > 1) return plan.seconds + 1e-6 < 0.95 * by_tiles ? plan.count : 0;
  const double read = 4e-6 + b / 3.9e12, slow = by_tiles > read ? by_tiles : read;
  return 9e-6 + b / 5.0e12 < 0.95 * slow ? 1 : 0;
}

// A few rows: the logits in planes and their gradient, or a product that ends in it, and
// both gradients in one reading of B (kernel_xent_few.hpp).
constexpr int64_t kFewRows = 16, kFewLogits = 8;   // of the gradients; of the logits

// A launch over B as it is stored, rows x cols.
struct FewGrid {
  int part, blocks, parts;
};

// Down: as many workgroups as their registers let reside, in one round (T = 8, H = 3271, V
// = 7145 V x H: 40 us, two rounds 44 and more planes to add up).  Across: 2048, so that
// they end together (8, 1024, 32768: 48; 1024 workgroups 54, 768 50).
FewGrid few_grid(bool down, bool grad, int64_t T, int64_t rows, int64_t cols) {
  const int64_t groups = !down ? 2048
                         : grad ? (T <= 1 ? 1280 : T <= 2 ? 1024 : T <= 4 ? 768 : 512)
                                : (T <= 4 ? 1280 : 768);
  const int64_t blocks = cdiv(cols, down ? 64 * sg::xent_few_cols((int)T) : 1024);
  int64_t part = round_up(cdiv(rows, at_least_one(groups / blocks)), down ? 32 : 8);
  if (!down && part > sg::kXentFewAcross) part = sg::kXentFewAcross;
  return {(int)part, (int)blocks, (int)cdiv(rows, part)};
}

// The logits that xent_few_down_kernel makes.
bool few_logits(bool trans_b, int64_t T, int64_t V, int64_t H) {
  return !trans_b && T > 0 && T <= kFewLogits && V > 0 && H > 0 && 4 * T * V <= kPlanesOne;
}

// Forward, where rows of B begin at any 4 bytes and B is beyond the caches (us, products /
// this: 4, 3144, 37682  165 / 99, 8, 4000, 20003  138 / 71, 1, 1100, 90001  88 / 83; smaller
// 7, 900, 30001  28 / 34, 1, 2000, 9999  27 / 32; aligned 2, 1786, 56588  83 / 85).
constexpr int64_t kFewForward = int64_t(256) << 20;   // bytes

struct Forward {
  const XentVariant* v;
  bool gathered;
  int strips;
  int planes;   // 0: by tiles
  FewGrid few;  // part 0: the planes are a product's
  XentRows rows;
  float *z, *max, *sum, *hit;
  int64_t bytes;
};

Forward plan_forward(bool trans_b, int64_t T, int64_t V, int64_t H, void* ws) {
  Forward f = {};
  f.v = choose(trans_b, T, V, H);
  if (f.v == nullptr) return f;
  f.gathered = 2.0 * T * V * H / 150e12 > kGatherSeconds && rows_fit(T, H);
  f.planes = f.gathered ? 0 : choose_planes(f.v, false, trans_b, T, V, H);
  if (!f.gathered && few_logits(trans_b, T, V, H) && V % 4 != 0 && 4 * V * H >= kFewForward) {
    f.few = few_grid(true, false, T, H, V);
    f.planes = f.few.parts;
  }
  f.strips = (int)cdiv(V, f.planes > 0 ? sg::kXentPlanesCols / 4 : f.v->strip);
  Room room = {static_cast<char*>(ws), 0};
  if (f.gathered) f.rows = take_rows(room, T, H, false);
  if (f.planes > 0) f.z = room.take<float>(f.planes * T * V);
  f.max = room.take<float>(f.strips * T);
  f.sum = room.take<float>(f.strips * T);
  f.hit = room.take<float>(T);
  f.bytes = room.used;
  return f;
}

// Backward, dZ of a piece takes at most this much where that leaves 1024 columns.
// Smaller ones cost more rounds of tiles and passes over dX (8192 tokens, H = 1024, V =
// 32768, with 128 MiB, 512 MiB and 1 GiB: 11.38, 11.17, 11.12 ms).
constexpr int64_t kPieceBytes = int64_t(512) << 20;
constexpr int64_t kPieceStep = 256;   // columns, the widest tile

int64_t piece_columns(int64_t T, int64_t V, int64_t bytes) {
  const int64_t n = T > 0 ? bytes / (4 * T) : V;
  return n >= V ? V : n / kPieceStep * kPieceStep;
}

struct Few {
  bool possible;
  FewGrid z, grad;   // z: by xent_few_down_kernel; part 0: by a product
  const XentVariant* v;   // that ends in dz; null: in planes
  int count;         // planes of dX
  int z_count;       // and of the logits
  float *z_planes, *planes;
  sg::XentRow* row;
  int64_t bytes;
};

Few plan_few(bool trans_b, int64_t T, int64_t V, int64_t H, void* ws) {
  Few f = {};
  if (T == 0 || T > kFewRows || V == 0 || H == 0 || 4 * T * V > kPlanesOne) return f;
  const int64_t rows = trans_b ? V : H, cols = trans_b ? H : V;
  f.grad = few_grid(trans_b, true, T, rows, cols);
  f.count = trans_b ? f.grad.parts : f.grad.blocks;
  if (few_logits(trans_b, T, V, H)) {
    f.z = few_grid(true, false, T, rows, cols);
    f.z_count = f.z.parts;
  } else {
    f.v = choose(trans_b, T, V, H);
    if (f.v == nullptr) return f;
    f.z_count = choose_planes(f.v, false, trans_b, T, V, H);
    if (f.z_count == 0) {
      // By rows, B read twice, where its tiles are too few (15, 4000, 600 V x H 30 us, tiles
      // 70; 16, 64, 60000 53 and 31).
      const PlanesPlan z = plan_planes(false, trans_b, T, V, H, kPlanesAll);
      const int64_t tiles = cdiv(T, f.v->cost.tile_m) * cdiv(V, f.v->cost.tile_n);
      if (z.possible && z.count == 1 && z.seconds < 0.5 * estimate_grid(f.v->cost, tiles, H))
        f.z_count = 1;
    }
    if (f.z_count > 0) f.v = nullptr;
    else f.z_count = 1;
  }
  if (!grid_fits((int64_t)f.grad.blocks * f.grad.parts, sg::kXentFewThreads)) return f;
  Room room = {static_cast<char*>(ws), 0};
  f.z_planes = room.take<float>(f.z_count * T * V);
  f.planes = room.take<float>(f.count * T * H);
  if (f.v) f.row = room.take<sg::XentRow>(T);
  f.bytes = room.used;
  f.possible = true;
  return f;
}

struct Backward {
  XentRows rows;
  float* dX;       // of the kept rows
  float* dZ;       // T x columns
  int planes;      // 0: by tiles; dZ is the first plane
  int64_t columns;
  int64_t fixed, bytes;   // without dZ; with it
  int64_t split;   // bytes the products take behind it for their fastest plans
};

// The plan for `bytes` of workspace, columns 0: too little; bytes < 0: the fastest.
Backward plan_backward(bool trans_b, int64_t T, int64_t V, int64_t H, void* ws, int64_t bytes) {
  Backward b = {};
  Room room = {static_cast<char*>(ws), 0};
  b.rows = take_rows(room, T, H, true);
  b.dX = room.take<float>(T * H);
  b.fixed = room.used;
  const int64_t least = 4 * at_least_one(T) * 1024;
  int64_t columns = piece_columns(T, V, kPieceBytes > least ? kPieceBytes : least);
  // What dZ may take, which ends on 16 bytes like every part.
  const int64_t left = bytes < 0 ? INT64_MAX : bytes > b.fixed ? (bytes - b.fixed) / 16 * 16 : 0;
  const int64_t most = piece_columns(T, V, left);
  if (most < columns) columns = most;
  // Equal pieces, of whole fours of tiles if they may be, which more often makes whole
  // rounds of them (16384 tokens, H = 512, V = 20000: 7.7 -> 7.4 ms).
  if (columns > 0 && columns < V) {
    const int64_t equal = cdiv(V, cdiv(V, columns));
    const int64_t four = round_up(equal, 4 * kPieceStep);
    columns = four <= columns ? four : round_up(equal, kPieceStep);
  }
  b.columns = columns;
  if (columns > 0 && T > 0) {
    b.planes = choose_planes(choose(trans_b, T, columns, H), true, trans_b, T, columns, H);
    if (left < 4 * b.planes * T * columns) b.planes = 0;
  }
  b.dZ = room.take<float>((b.planes > 1 ? b.planes : 1) * T * columns);
  b.bytes = room.used;
  const int64_t x = sgemm_grouped_workspace_bytes(!trans_b, T, H, columns, 1);
  const int64_t w = sgemm_grouped_wgrad_workspace_bytes(trans_b, T, columns, H, 1);
  b.split = x > w ? x : w;
  return b;
}

int launch(const void* fn, int64_t wgs, int threads, void* args, hipStream_t stream) {
  void* kargs[] = {args};
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(threads), kargs, 0, stream) == hipSuccess
             ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

// The rows with a target numbered and copied together.
int gather(const Targets& targets, const XentRows& rows, int64_t T, int64_t H, const float* X,
           int64_t ldx, const float* lse, const float* dloss, hipStream_t stream) {
  XentPlaceArgs a = {};
  a.targets = targets;
  a.rows = rows;
  a.lse = lse;
  a.dloss = dloss;
  a.T = T;
  if (T > 0 && T <= sg::kXentGatherRows) {
    a.X = X;
    a.ldx = ldx;
    a.H = (int)H;
    const int64_t waves = T * at_least_one(cdiv(H, sg::kXentGatherCols));
    return launch(reinterpret_cast<const void*>(sg::xent_gather_kernel), cdiv(waves, 4), 256, &a,
                  stream);
  }
  // Up to 256 workgroups, as each reads all the targets before its own.
  a.chunk = round_up(at_least_one(cdiv(T, 256)), sg::kXentPlaceThreads);
  const int st = launch(reinterpret_cast<const void*>(sg::xent_place_kernel),
                        at_least_one(cdiv(T, a.chunk)), sg::kXentPlaceThreads, &a, stream);
  return st != SGEMM_OK ? st : sgemm_moe_permute(T, 1, H, X, ldx, rows.place, rows.X,
                                                 at_least_one(H), stream);
}

// Tiles of columns column .. column + V - 1 of op(B).
int launch_product(const XentVariant& v, XentProductArgs& a, bool grad, hipStream_t stream) {
  const TileCost& c = v.cost;
  a.tiles_m = (int)cdiv(a.M, c.tile_m);
  a.tiles_n = (int)cdiv(a.N, c.tile_n);
  a.group_m = a.tiles_m < 8 ? a.tiles_m : 8;
  a.splits = 1;
  a.turn = a.tiles_m == 1;   // bound by reading B (two rows of tiles: no difference)
  return launch(reinterpret_cast<const void*>(grad ? v.grad : v.stats),
                (int64_t)a.tiles_m * a.tiles_n, c.threads, &a, stream);
}

XentProductArgs product_args(int64_t T, int64_t V, int64_t H, const float* X, int64_t ldx,
                             const float* B, int64_t ldb, const int32_t* offsets) {
  XentProductArgs a;
  memset(&a, 0, sizeof(a));
  a.A = X;
  a.B = B;
  a.M = (int)T;
  a.N = (int)V;
  a.K = (int)H;
  a.lda = (int)ldx;
  a.ldb = (int)ldb;
  a.ldc = 1;
  a.mode = offsets ? sg::kRowGroups : sg::kDense;
  a.groups = 1;
  a.rows = (int)T;
  a.offsets = offsets;
  return a;
}

// A kernel of the least rows that hold T.
enum class FewKernel { kLogits, kDown, kAcross };

template <int R>
const void* few_kernel(FewKernel which, int64_t T) {
  if constexpr (R < kFewRows)
    if (T > R) return few_kernel<2 * R>(which, T);
  if constexpr (R <= kFewLogits)
    if (which == FewKernel::kLogits)
      return reinterpret_cast<const void*>(sg::xent_few_down_kernel<R, false>);
  if (which == FewKernel::kDown)
    return reinterpret_cast<const void*>(sg::xent_few_down_kernel<R, true>);
  return reinterpret_cast<const void*>(sg::xent_few_across_kernel<R>);
}

int launch_few(FewKernel which, const FewGrid& grid, XentFewArgs& a, hipStream_t stream) {
  a.part = grid.part;
  a.blocks = grid.blocks;
  return launch(few_kernel<1>(which, a.T), (int64_t)grid.blocks * grid.parts, sg::kXentFewThreads,
                &a, stream);
}

// Checks of both calls: sizes, leading dimensions, targets.
int check(int trans_b, int64_t T, int64_t V, int64_t H, int64_t ldx, int64_t ldb, int id_bytes,
          const void* targets, int64_t ws_bytes) {
  if ((trans_b & ~1) || T < 0 || V < 0 || H < 0 || ldx < at_least_one(H) ||
      ldb < at_least_one(trans_b ? H : V) || (id_bytes != 4 && id_bytes != 8) || ws_bytes < 0 ||
      ((uintptr_t)targets & (uintptr_t)(id_bytes - 1)))
    return SGEMM_ERR_INVALID_ARG;
  if (!sizes_ok(T, V, H) || leading(T, H, ldx) > SGEMM_XENT_MAX_LD ||
      leading(trans_b ? V : H, trans_b ? H : V, ldb) > SGEMM_XENT_MAX_LD)
    return SGEMM_ERR_UNSUPPORTED;
  return SGEMM_OK;
}

}  // namespace

extern "C" {

int64_t sgemm_linear_xent_workspace_bytes(int trans_b, int64_t T, int64_t V, int64_t H) {
  if ((trans_b & ~1) || !sizes_ok(T, V, H) || T == 0) return 0;
  return plan_forward(trans_b, T, V, H, nullptr).bytes;
}

int sgemm_linear_xent(int trans_b, int64_t T, int64_t V, int64_t H, const float* X, int64_t ldx,
                      const float* B, int64_t ldb, const void* targets, int id_bytes, float* loss,
                      float* lse, hipStream_t stream, void* workspace, int64_t workspace_bytes) {
  int st = check(trans_b, T, V, H, ldx, ldb, id_bytes, targets, workspace_bytes);
  if (st == SGEMM_ERR_INVALID_ARG) return st;
  if (T == 0) return st;
  const Span in[] = {{X, V > 0 ? span_bytes(T, H, ldx) : 0},
                     {B, trans_b ? span_bytes(V, H, ldb) : span_bytes(H, V, ldb)},
                     {targets, T * id_bytes}};
  const Span out[] = {{loss, 4 * T}, {lse, lse ? 4 * T : 0}};
  for (const Span& s : in)
    if (bad(s)) return SGEMM_ERR_INVALID_ARG;
  for (const Span& s : out)
    if (bad(s)) return SGEMM_ERR_INVALID_ARG;
  if (st != SGEMM_OK) return st;
  const Forward f = plan_forward(trans_b, T, V, H, workspace);
  const int rows = T >= kLossRowsFrom ? 32 : 16;   // a workgroup of xent_loss_kernel
  if (f.v == nullptr || !grid_fits(cdiv(T, rows), sg::kXentLossThreads))
    return SGEMM_ERR_UNSUPPORTED;
  const Span ws = {workspace, f.bytes};
  if (workspace_bytes < f.bytes || bad(ws)) return SGEMM_ERR_INVALID_ARG;
  for (const Span& s : in)
    if (overlaps(s, out[0]) || overlaps(s, out[1]) || overlaps(s, ws)) return SGEMM_ERR_INVALID_ARG;
  if (overlaps(out[0], out[1]) || overlaps(out[0], ws) || overlaps(out[1], ws))
    return SGEMM_ERR_INVALID_ARG;

  ldx = leading(T, H, ldx);
  ldb = leading(trans_b ? V : H, trans_b ? H : V, ldb);
  const Targets t = {targets, id_bytes == 8, (int)V};
  if (V > 0 && f.gathered)
    st = gather(t, f.rows, T, H, X, ldx, nullptr, nullptr, stream);
  if (V > 0 && st == SGEMM_OK && f.planes > 0) {
    XentPlanesArgs a = {};
    if (f.few.part > 0) {
      XentFewArgs l = {};
      l.targets = t;
      l.B = B;
      l.P = X;
      l.planes = f.z;
      l.T = (int)T;
      l.rows = (int)H;
      l.cols = (int)V;
      l.ldb = (int)ldb;
      l.ldp = (int)ldx;
      a.count = f.planes;
      st = launch_few(FewKernel::kLogits, f.few, l, stream);
    } else {
      st = launch_planes(trans_b, T, V, H, X, ldx, B, ldb, nullptr, f.z, 4 * f.planes * T * V,
                         stream, a.count);
    }
    a.planes = f.z;
    a.targets = t;
    a.max = f.max;
    a.sum = f.sum;
    a.hit = f.hit;
    a.rows = (int)T;
    a.N = (int)V;
    if (st == SGEMM_OK)
      st = launch(reinterpret_cast<const void*>(sg::xent_planes_stats_kernel),
                  T * cdiv(V, sg::kXentPlanesCols), 256, &a, stream);
  } else if (V > 0 && st == SGEMM_OK) {
    XentProductArgs a = f.gathered
                            ? product_args(T, V, H, f.rows.X, at_least_one(H), B, ldb, f.rows.offsets)
                            : product_args(T, V, H, X, ldx, B, ldb, nullptr);
    a.targets = t;
    a.target = f.gathered ? f.rows.target : nullptr;
    a.max = f.max;
    a.sum = f.sum;
    a.hit = f.hit;
    a.ld_strip = (int)T;
    st = launch_product(*f.v, a, false, stream);
  }
  if (st != SGEMM_OK) return st;
  XentLossArgs l = {};
  l.targets = t;
  l.place = f.gathered ? f.rows.place : nullptr;
  l.max = f.max;
  l.sum = f.sum;
  l.hit = f.hit;
  l.loss = loss;
  l.lse = lse;
  l.T = T;
  l.strips = f.strips;
  l.ld_strip = (int)T;
  return launch(rows == 32 ? reinterpret_cast<const void*>(sg::xent_loss_kernel<32>)
                           : reinterpret_cast<const void*>(sg::xent_loss_kernel<16>),
                cdiv(T, rows), sg::kXentLossThreads, &l, stream);
}

int64_t sgemm_linear_xent_backward_workspace_bytes(int trans_b, int64_t T, int64_t V, int64_t H) {
  if ((trans_b & ~1) || !sizes_ok(T, V, H)) return 0;
  const Backward b = plan_backward(trans_b, T, V, H, nullptr, -1);
  const Few f = plan_few(trans_b, T, V, H, nullptr);
  if (!f.possible) return b.bytes + b.split;
  const int64_t least = sgemm_linear_xent_backward_least_bytes(trans_b, T, V, H);
  return f.bytes > least ? f.bytes : least;
}

int64_t sgemm_linear_xent_backward_least_bytes(int trans_b, int64_t T, int64_t V, int64_t H) {
  if ((trans_b & ~1) || !sizes_ok(T, V, H)) return 0;
  const Backward b = plan_backward(trans_b, T, V, H, nullptr, -1);
  return b.fixed + round_up(4 * T * (V < kPieceStep ? V : kPieceStep), 16);
}

int sgemm_linear_xent_backward(int trans_b, int64_t T, int64_t V, int64_t H, const float* X,
                               int64_t ldx, const float* B, int64_t ldb, const void* targets,
                               int id_bytes, const float* lse, const float* dloss, float* dX,
                               int64_t lddx, float* dB, int64_t lddb, hipStream_t stream,
                               void* workspace, int64_t workspace_bytes) {
  int st = check(trans_b, T, V, H, ldx, ldb, id_bytes, targets, workspace_bytes);
  if (st == SGEMM_ERR_INVALID_ARG || (dX && lddx < at_least_one(H)) ||
      (dB && lddb < at_least_one(trans_b ? H : V)))
    return SGEMM_ERR_INVALID_ARG;
  if (H == 0 || (!dX && !dB)) return st;
  const int64_t br = trans_b ? V : H, bc = trans_b ? H : V;
  const Span in[] = {{X, V > 0 ? span_bytes(T, H, ldx) : 0},
                     {B, span_bytes(br, bc, ldb)},
                     {targets, T * id_bytes},
                     {lse, 4 * T},
                     {dloss, 4 * T}};
  const Span out[] = {{dX, dX ? span_bytes(T, H, lddx) : 0}, {dB, dB ? span_bytes(br, bc, lddb) : 0}};
  for (const Span& s : in)
    if (bad(s)) return SGEMM_ERR_INVALID_ARG;
  for (const Span& s : out)
    if (bad(s)) return SGEMM_ERR_INVALID_ARG;
  if (st != SGEMM_OK) return st;
  if (out[0].bytes < 0 || (dB && leading(br, bc, lddb) > SGEMM_XENT_MAX_LD))
    return SGEMM_ERR_UNSUPPORTED;
  const Backward b = plan_backward(trans_b, T, V, H, workspace, workspace_bytes);
  if (V > 0 && (b.columns == 0 || workspace_bytes < b.bytes)) return SGEMM_ERR_INVALID_ARG;
  if (workspace_bytes < b.fixed) return SGEMM_ERR_INVALID_ARG;
  const Few f = plan_few(trans_b, T, V, H, workspace);
  const bool few = f.possible && f.bytes <= workspace_bytes;
  int64_t used = few ? f.bytes : b.bytes + b.split;
  if (used > workspace_bytes) used = workspace_bytes;
  const Span ws = {workspace, used};
  if (bad(ws)) return SGEMM_ERR_INVALID_ARG;
  for (const Span& s : in)
    if (overlaps(s, out[0]) || overlaps(s, out[1]) || overlaps(s, ws)) return SGEMM_ERR_INVALID_ARG;
  if (overlaps(out[0], out[1]) || overlaps(out[0], ws) || overlaps(out[1], ws))
    return SGEMM_ERR_INVALID_ARG;
  const XentVariant* v = V > 0 ? choose(trans_b, T, b.columns, H) : nullptr;
  if ((V > 0 && v == nullptr) || !rows_fit(T, H)) return SGEMM_ERR_UNSUPPORTED;

  ldx = leading(T, H, ldx);
  ldb = leading(br, bc, ldb);
  if (dB) lddb = leading(br, bc, lddb);
  const Targets t = {targets, id_bytes == 8, (int)V};
  if (few) {
    XentFewArgs a = {};
    a.targets = t;
    a.B = B;
    a.T = (int)T;
    a.rows = (int)br;
    a.cols = (int)bc;
    a.ldb = (int)ldb;
    if (f.v) {
      XentPlaceArgs p = {};
      p.targets = t;
      p.rows.row = f.row;
      p.lse = lse;
      p.dloss = dloss;
      p.T = T;
      st = launch(reinterpret_cast<const void*>(sg::xent_rows_kernel), 1, 64, &p, stream);
      if (st != SGEMM_OK) return st;
      XentProductArgs z = product_args(T, V, H, X, ldx, B, ldb, nullptr);
      z.C = f.z_planes;
      z.ldc = (int)V;
      z.row = f.row;
      st = launch_product(*f.v, z, true, stream);
    } else {
      XentPlanesArgs p = {};
      if (f.z.part == 0) {
        st = launch_planes(trans_b, T, V, H, X, ldx, B, ldb, nullptr, f.z_planes, kPlanesAll,
                           stream, p.count);
      } else {
        p.count = f.z_count;
        a.P = X;
        a.ldp = (int)ldx;
        a.planes = f.z_planes;
        st = launch_few(FewKernel::kLogits, f.z, a, stream);
      }
      if (st != SGEMM_OK) return st;
      p.planes = f.z_planes;
      p.dZ = f.z_planes;
      p.targets = t;
      p.lse = lse;
      p.dloss = dloss;
      p.rows = (int)T;
      p.N = (int)V;
      st = launch(reinterpret_cast<const void*>(sg::xent_planes_grad_kernel),
                  T * cdiv(V, sg::kXentPlanesCols), 256, &p, stream);
    }
    if (st != SGEMM_OK) return st;
    a.P = trans_b ? f.z_planes : X;
    a.ldp = (int)(trans_b ? V : ldx);
    a.Q = trans_b ? X : f.z_planes;
    a.ldq = (int)(trans_b ? ldx : V);
    a.D = dB;
    a.ldd = dB ? (int)lddb : 0;
    a.planes = dX ? f.planes : nullptr;
    st = launch_few(trans_b ? FewKernel::kDown : FewKernel::kAcross, f.grad, a, stream);
    if (st != SGEMM_OK || !dX) return st;
    XentFewSumArgs sum = {t, f.planes, dX, leading(T, H, lddx), (int)T, (int)H, f.count};
    return launch(reinterpret_cast<const void*>(sg::xent_few_sum_kernel),
                  T * cdiv(H, sg::kXentFewSumCols), sg::kXentFewThreads, &sum, stream);
  }
  const XentRows& r = b.rows;
  st = gather(t, r, T, V > 0 ? H : 0, X, ldx, lse, dloss, stream);
  char* const split = static_cast<char*>(workspace) + b.bytes;
  const int64_t split_bytes = used - b.bytes;
  for (int64_t c0 = 0; c0 < V && st == SGEMM_OK; c0 += b.columns) {
    const int64_t n = V - c0 < b.columns ? V - c0 : b.columns;
    const float* const Bp = B + (trans_b ? c0 * ldb : c0);
    const int64_t ldz = b.planes > 0 ? n : b.columns;
    if (b.planes > 0) {
      XentPlanesArgs a = {};
      st = launch_planes(trans_b, T, n, H, r.X, H, Bp, ldb, r.offsets, b.dZ,
                         4 * b.planes * T * b.columns, stream, a.count);
      a.planes = b.dZ;
      a.dZ = b.dZ;
      a.offsets = r.offsets;
      a.row = r.row;
      a.rows = (int)T;
      a.N = (int)n;
      a.column0 = (int)c0;
      if (st == SGEMM_OK)
        st = launch(reinterpret_cast<const void*>(sg::xent_planes_grad_kernel),
                    T * cdiv(n, sg::kXentPlanesCols), 256, &a, stream);
    } else if (T > 0) {
      XentProductArgs a = product_args(T, n, H, r.X, H, Bp, ldb, r.offsets);
      a.C = b.dZ;
      a.ldc = (int)ldz;
      a.row = r.row;
      a.column0 = (int)c0;
      st = launch_product(*v, a, true, stream);
    }
    if (st == SGEMM_OK && dB)
      st = sgemm_grouped_wgrad(trans_b, T, n, H, 1, r.offsets, r.X, H, b.dZ, ldz,
                               dB + (trans_b ? c0 * lddb : c0), lddb,
                               span_bytes(trans_b ? n : H, trans_b ? H : n, lddb) / 4, stream,
                               split, split_bytes);
    if (st == SGEMM_OK && dX && T > 0) {
      // The pieces' parts of dX add up in place.
      sgemm_epilogue add = {};
      add.residual = c0 > 0 ? b.dX : nullptr;
      add.ldr = H;
      st = sgemm_grouped(!trans_b, T, H, n, 1, r.offsets, b.dZ, ldz, Bp, ldb,
                         span_bytes(trans_b ? n : H, trans_b ? H : n, ldb) / 4, b.dX, H, &add,
                         stream, split, split_bytes);
    }
  }
  if (st == SGEMM_OK && dX && T > 0)
    st = sgemm_moe_unpermute(T, 1, H, b.dX, H, r.place, nullptr, dX, lddx, stream);
  return st;
}

}  // extern "C"
