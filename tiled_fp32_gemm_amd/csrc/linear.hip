// linear.hip -- the C ABI of include/sgemm_linear.h and the grouped products of
// include/sgemm_moe.h: argument checks, kernel choice and launch.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../include/sgemm_linear.h"
#include "../../include/sgemm_moe.h"
#include "host.hpp"
#include "kernel_act_backward.hpp"
#include "kernel_product_reduce.hpp"
#include "product_variants.hpp"

namespace {

using namespace sg::host;
using sg::ActBackwardArgs;
using sg::ProductArgs;

using sg::ProductVariant;

struct Span {
  const void* p;
  int64_t bytes;   // 0: not touched; -1: beyond int64
};

// A span that is touched has to be there and aligned; one beyond int64 is
// unsupported.
int check_spans(const Span* s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i].bytes != 0 && (s[i].p == nullptr || ((uintptr_t)s[i].p & 3u)))
      return SGEMM_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (s[i].bytes < 0) return SGEMM_ERR_UNSUPPORTED;
  return SGEMM_OK;
}

bool overlaps(const Span& a, const Span& b) {
  return sg::host::overlaps(a.p, a.bytes, b.p, b.bytes);
}

int64_t at_least_one(int64_t n) { return n > 1 ? n : 1; }

// Bytes of n floats; -1 where n is past any limit.
int64_t floats(int64_t n) { return n > kMaxDim ? -1 : 4 * n; }

// A leading dimension as the kernels take it: it only matters past the first
// row.  -1: more than an int.
int leading(int64_t rows, int64_t width, int64_t ld) {
  const int64_t n = rows > 1 ? ld : at_least_one(width);
  return n > INT32_MAX ? -1 : (int)n;
}

// Bytes of `groups` matrices of `one` bytes, `stride` floats apart.
int64_t groups_bytes(int64_t groups, int64_t stride, int64_t one) {
  if (groups == 0 || one <= 0) return groups == 0 ? 0 : one;
  if (groups - 1 > (INT64_MAX / 4 - one) / at_least_one(stride)) return -1;
  return (groups - 1) * stride * 4 + one;
}

// The operands of one call, checked.
struct Product {
  ProductArgs g;
  bool trans_a, trans_b;
  bool launch;   // false: nothing to do
  Span a, b, c, bias, res, pre;
};

// Checks that hold for every kind: sizes, leading dimensions, epilogue,
// pointers, overlaps.  Groups: stride_b (kRowGroups) or stride_c (kSumGroups).
int check_product(int mode, int ta, int tb, int64_t M, int64_t N, int64_t K, int64_t groups,
                  const int32_t* offsets, int64_t rows, const float* A, int64_t lda,
                  const float* B, int64_t ldb, int64_t stride_b, float* C, int64_t ldc,
                  int64_t stride_c, const sgemm_epilogue* ep, const void* ws, int64_t ws_bytes,
                  Product& p) {
  memset(&p, 0, sizeof(p));
  if ((ta | tb) & ~1) return SGEMM_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K < 0 || rows < 0 || groups < 0) return SGEMM_ERR_INVALID_ARG;
  if (ws_bytes < 0 || (ws_bytes > 0 && ws == nullptr) || ((uintptr_t)ws & 3u))
    return SGEMM_ERR_INVALID_ARG;
  const int64_t ar = ta ? K : M, ac = ta ? M : K, br = tb ? N : K, bc = tb ? K : N;
  if (lda < at_least_one(ac) || ldb < at_least_one(bc) || ldc < at_least_one(N))
    return SGEMM_ERR_INVALID_ARG;
  static const sgemm_epilogue none = {};
  if (ep == nullptr) ep = &none;
  if (ep->act < SGEMM_ACT_NONE || ep->act > SGEMM_ACT_SILU) return SGEMM_ERR_INVALID_ARG;
  if ((ep->residual && ep->ldr < at_least_one(N)) || (ep->preact && ep->ldp < at_least_one(N)) ||
      (mode == sg::kRowGroups && ep->bias && ep->ldbias < at_least_one(N)))
    return SGEMM_ERR_INVALID_ARG;
  if (groups > sg::kMaxGroups) return SGEMM_ERR_UNSUPPORTED;

  const bool touch = M > 0 && N > 0 && (mode == sg::kDense || groups > 0);
  p.launch = touch;
  if (!touch) return SGEMM_OK;
  const bool sums = mode == sg::kSumGroups;
  p.a = {A, span_bytes(ar, ac, lda)};
  p.b = {B, span_bytes(br, bc, ldb)};
  p.c = {C, span_bytes(M, N, ldc)};
  p.res = {ep->residual, ep->residual ? span_bytes(M, N, ep->ldr) : 0};
  p.pre = {ep->preact, ep->preact ? span_bytes(M, N, ep->ldp) : 0};
  p.bias = {ep->bias, !ep->bias                ? 0
                      : mode == sg::kRowGroups ? groups_bytes(groups, ep->ldbias, floats(N))
                                               : floats(N)};
  if (mode == sg::kRowGroups) {
    if (p.b.bytes > 0 && groups > 1 && stride_b < p.b.bytes / 4) return SGEMM_ERR_INVALID_ARG;
    p.b.bytes = groups_bytes(groups, stride_b, p.b.bytes);
  }
  if (sums) {
    if (p.c.bytes > 0 && groups > 1 && stride_c < p.c.bytes / 4) return SGEMM_ERR_INVALID_ARG;
    p.c.bytes = groups_bytes(groups, stride_c, p.c.bytes);
  }
  const Span off = {offsets, mode == sg::kDense ? 0 : (groups + 1) * 4};
  const Span all[] = {p.a, p.b, p.c, p.bias, p.res, p.pre, off};
  const int st = check_spans(all, 7);
  if (st != SGEMM_OK) return st;
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim || rows > kMaxDim) return SGEMM_ERR_UNSUPPORTED;
  const bool in_place = ep->residual == C && ep->ldr == ldc;
  if (overlaps(p.c, p.a) || overlaps(p.c, p.b) || overlaps(p.c, p.bias) ||
      overlaps(p.c, p.pre) || overlaps(p.c, off) || (!in_place && overlaps(p.c, p.res)) ||
      overlaps(p.pre, p.a) || overlaps(p.pre, p.b) || overlaps(p.pre, p.bias) ||
      overlaps(p.pre, p.res) || overlaps(p.pre, off))
    return SGEMM_ERR_INVALID_ARG;

  ProductArgs& g = p.g;
  p.trans_a = ta;
  p.trans_b = tb;
  g.A = A;
  g.B = B;
  g.C = C;
  g.M = (int)M;
  g.N = (int)N;
  g.K = (int)K;
  g.lda = leading(K > 0 ? ar : 0, ac, lda);
  g.ldb = leading(K > 0 ? br : 0, bc, ldb);
  g.ldc = leading(M, N, ldc);
  g.bias = ep->bias;
  g.residual = ep->residual;
  g.preact = ep->preact;
  g.ld_bias = ep->ldbias;
  g.ldr = ep->residual ? leading(M, N, ep->ldr) : 1;
  g.ldp = ep->preact ? leading(M, N, ep->ldp) : 1;
  if (g.lda < 0 || g.ldb < 0 || g.ldc < 0 || g.ldr < 0 || g.ldp < 0) return SGEMM_ERR_UNSUPPORTED;
  g.act = ep->act;
  g.mode = mode;
  g.groups = mode == sg::kDense ? 1 : (int)groups;
  g.rows = (int)rows;
  g.offsets = offsets;
  g.stride_b = stride_b;
  g.stride_c = stride_c;
  g.splits = 1;
  return SGEMM_OK;
}

const ProductVariant* variants(bool trans_a, bool trans_b) {
  if (trans_a) return trans_b ? sg::product_variants_sf() : sg::product_variants_ss();
  return trans_b ? sg::product_variants_ff() : sg::product_variants_fs();
}

// Whether a variant's 32-bit offsets reach its tile's part of every operand:
// with k running along the rows all of k, with k from row to row one slab.
bool variant_fits(const Product& p, const ProductVariant& v) {
  const ProductArgs& g = p.g;
  const sg::host::TileCost& c = v.cost;
  const int64_t K = g.mode == sg::kSumGroups ? c.tile_k : g.K;
  auto fits = [&](bool k_fast, int64_t extent, int tile, int64_t ld) {
    if (K == 0) return true;
    return k_fast ? span_fits(extent < tile ? extent : tile, K > c.tile_k ? K : c.tile_k, ld)
                  : span_fits(K < c.tile_k ? K : c.tile_k, tile, ld);
  };
  const int64_t rows = g.M < c.tile_m ? g.M : c.tile_m;
  return fits(!p.trans_a, g.M, c.tile_m, g.lda) && fits(p.trans_b, g.N, c.tile_n, g.ldb) &&
         span_fits(rows, c.tile_n, g.ldc) &&
         (!g.residual || span_fits(rows, c.tile_n, g.ldr)) &&
         (!g.preact || span_fits(rows, c.tile_n, g.ldp)) && span_fits(rows, c.tile_n, g.N);
}

struct Choice {
  const ProductVariant* v;
  int splits, k_split;
  int64_t workgroups;   // of the grid
  double seconds;       // estimated
};

// Groups that can have rows.
int64_t live_groups(const ProductArgs& g) { return g.groups < g.M ? g.groups : g.M; }

// Workgroups of one split: exactly the tiles, except over row groups, whose
// tiles only the device can count; this is the most there can be.
int64_t grid_tiles(const ProductArgs& g, const sg::host::TileCost& c) {
  const int64_t tn = cdiv(g.N, c.tile_n);
  if (g.mode == sg::kRowGroups) {
    const int64_t live = live_groups(g);
    return ((g.M - live) / c.tile_m + live) * tn;
  }
  return cdiv(g.M, c.tile_m) * tn * g.groups;
}

// The estimate for `level` tiles on the busiest CU, between whole numbers of them.
double estimate_level(const sg::host::TileCost& c, double level, int64_t K) {
  const int64_t n = level < 1 ? 1 : (int64_t)level;
  const double less = estimate_grid(c, n * kCUs, K);
  return level <= n ? less : less + (level - n) * (estimate_grid(c, (n + 1) * kCUs, K) - less);
}

// Estimated seconds of a grid in `splits` parts of K each.  The lengths of
// groups are not known here, and their tiles are handed out as workgroups end:
// row groups are taken as 0.4, 0.7, 1, 1.3 and 1.6 times the average, which gives
// the tiles and, in a wave's rows (waves without rows leave the others their
// share), the work; the busiest CU has its share of the work and a part of a
// tile more.  Summed groups: the same, or, in one round, the longest.  The
// figures are fitted to 24 sets of uneven groups, 16 to 65536 rows in 4 to 128
// of them: the choice is 1.6% behind the fastest on average, 20% at worst.
double likely_time(const ProductArgs& g, const sg::host::TileCost& c, int64_t splits, int64_t K) {
  const int64_t tiles = grid_tiles(g, c) * splits;
  if (g.mode == sg::kDense || g.groups <= 1 || tiles == 0) return estimate_grid(c, tiles, K);
  if (g.mode == sg::kSumGroups)
    return tiles <= kCUs ? 1.2 * estimate_grid(c, tiles, K)
                         : estimate_level(c, (double)tiles / kCUs + (g.groups <= 16 ? 0.6 : 1.0), K);
  const int64_t live = live_groups(g), wave_rows = c.tile_m >= 256 ? 64 : 32;
  int64_t likely = 0, waves = 0;   // of five groups
  for (int i = 4; i <= 16; i += 3) {
    const int64_t rows = cdiv((int64_t)g.M * i, 10 * live);
    likely += cdiv(rows, c.tile_m);
    waves += cdiv(rows, wave_rows);
  }
  const double all = (double)live / 5.0 * (double)(cdiv(g.N, c.tile_n) * splits);
  const double more = c.tile_m >= 128 ? 1.2 : c.tile_m >= 64 ? 1.16 : 1.06;
  const double count = 1.13 * all * likely, work = more * all * waves * wave_rows / c.tile_m;
  if (count <= kCUs) return estimate_grid(c, (int64_t)count, K);
  const double level = work / kCUs + (c.tile_m >= 128 ? 0.3 : 0.4);
  const double most = (double)cdiv((int64_t)count, kCUs);
  return estimate_level(c, level < most ? level : most, K);
}

// What a split costs beside its tiles and its planes' traffic, fitted with the
// tiles' figures: the part of a grid's time that remains when it need not end
// with C, a second launch, and that one's wait for each plane.
constexpr double kSplitPart = 0.93, kSplitFixed = 3.5e-6, kSplitPlane = 0.08e-6;

// The variant, and the split of K, with the least estimated time (the model
// of host.hpp).  A null v: no variant can address this product.
Choice choose(const Product& p, int64_t ws_bytes) {
  const ProductArgs& g = p.g;
  const ProductVariant* table = variants(p.trans_a, p.trans_b);
  // kSumGroups: the sum's length, groups taken as equal.
  const int64_t K = g.mode == sg::kSumGroups ? cdiv(g.rows, at_least_one(g.groups)) : g.K;
  const int64_t out = (int64_t)g.M * g.N * (g.mode == sg::kSumGroups ? g.groups : 1);
  Choice one = {nullptr, 1, 0, 0, 0.0}, split = one;
  double t_one = 0, t_split = 0;
  static const int kSplits[] = {2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
  for (int i = 0; i < sg::kProductVariants; ++i) {
    const ProductVariant& v = table[i];
    const int64_t grid = grid_tiles(g, v.cost);
    if (!variant_fits(p, v) || !grid_fits(grid, v.cost.threads)) continue;
    const double t = likely_time(g, v.cost, 1, K);
    if (one.v == nullptr || t < t_one * 0.995) {
      one = {&v, 1, 0, grid, t};
      t_one = t;
    }
  }
  // A split takes the fixed costs of a round and of a second launch at least.
  if (one.v == nullptr || t_one < kRoundCost + kSplitFixed || 2 * out > ws_bytes / 4) return one;
  for (int i = 0; i < sg::kProductVariants; ++i) {
    const ProductVariant& v = table[i];
    const sg::host::TileCost& c = v.cost;
    const int64_t grid = grid_tiles(g, c);
    if (K < 2 * c.tile_k || !variant_fits(p, v)) continue;
    for (int S : kSplits) {
      // Few tiles and a long K: 64 x 64 x 65536 in 32 splits 29.1 us, in 64 22.9; the
      // second pass waits longer for more planes (64 x 64 x 16384: 14.0 with both).
      if (S > 32 && 32 * grid >= kCUs) break;
      const int64_t ks = cdiv(cdiv(K, S), c.tile_k) * c.tile_k;
      const int64_t se = g.mode == sg::kSumGroups ? S : cdiv(K, ks);
      if (se < 2 || se * out > ws_bytes / 4 || !grid_fits(grid * se, c.threads) ||
          !grid_fits(out / g.N * cdiv(g.N, sg::kProductReduceCols), 64))
        continue;
      const double ts = kSplitPart * likely_time(g, c, se, ks) + kSplitFixed +
                        kSplitPlane * se + (double)(se + 1) * out * 4.0 / kReduceBW;
      if (split.v == nullptr || ts < t_split) {
        split = {&v, (int)se, (int)ks, grid * se, ts};
        t_split = ts;
      }
    }
  }
  return split.v != nullptr && t_split < t_one * 0.95 ? split : one;
}

int64_t split_bytes(const ProductArgs& g, const Choice& ch) {
  if (ch.v == nullptr || ch.splits == 1) return 0;
  return (int64_t)ch.splits * g.M * g.N * (g.mode == sg::kSumGroups ? g.groups : 1) * 4;
}

// The kernels for a few rows (kernel_rows.hpp): rows a chunk, columns a
// workgroup; rows 0: not for this product.
struct RowsChoice {
  int rows, cols, threads;
  int64_t workgroups;
};

// Measured on MI355X against product_kernel with a workspace (us, rows /
// product; B from HBM, the groups' rows drawn at random, E x K x N):
//      B stored                 N x K                       K x N
//      1 row, 4096 x 4096    12.8 / 19.5                 18.2 / 21.8
//      4 rows                13.1 / 19.5                 19.2 / 20.9
//      8 rows                16.5 / 19.5                 21.0 / 20.8
//      16 rows               22.0 / 19.8                 22.3 / 21.1
//      8 rows, 11008 x 4096  36.9 / 43.9                 40.1 / 42.0
//      1 row, 4096 x 11008   30.4 / 47.9                 44.1 / 40.0
//      16 rows, 8192 x 1024  13.4 / 14.1                 12.2 / 13.8
//      16 rows, 2048 x 2048  10.5 / 11.3                 10.1 / 11.2
//      groups, on average    2       4       6            2       3       4
//      8 x 1024 x 4096     23/32   28/34   33/36        23/28   26/28   27/29
//      8 x 4096 x 1024     23/27   27/30   39/31        27/27   28/30   29/32
//      16 x 2048 x 2048    41/51   51/57   64/61        40/45   45/46   50/48
//      64 x 1024 x 1024    41/59   52/64   60/67        42/46   53/50   54/52
// Without room to split, up to 16 rows are the faster way unless the product's
// own tiles fill half the chip (16 rows, N = 4096: 22 / 50, N = 11008: 64 / 56).
// Columns a workgroup, K x N: the most that still give 5/8 of the CUs one, and
// eight waves for fewer than two a CU (4 rows, us, at 16, 32 and 64 columns with
// four / eight waves: N = K = 4096 20.1 / 19.1, 25.4 / 20.8, 43 / 27; 11008 x 4096
// 55 / 43, 45 / 49, 48 / 34; 32768 x 1024 32 / 33, 28 / 27, 21.6 / 22.5).
RowsChoice choose_rows(const Product& p) {
  const ProductArgs& g = p.g;
  RowsChoice none = {0, 0, 0, 0};
  // The kernels count k in ints, some way past K; a row that long is refused by
  // product_kernel's spans as well.
  if (p.trans_a || g.mode == sg::kSumGroups || g.K >= 1 << 29) return none;
  const bool grouped = g.mode == sg::kRowGroups;
  const int64_t live = grouped ? live_groups(g) : 1;
  const int64_t average = p.trans_b ? (g.N >= g.K ? 6 : 4) : live <= 8 ? 4 : 3;
  const int64_t most = grouped ? average * live : 2 * sg::kRowsMost;
  if (g.M > most && g.M > sg::kRowsMost) return none;
  // A chunk has room for a group of twice the average.
  const int64_t want = grouped ? cdiv(2 * g.M, live) : g.M;
  RowsChoice ch = {1, p.trans_b ? 16 : 64, 256, 0};
  while (ch.rows < sg::kRowsMost && ch.rows < want && ch.rows < g.M) ch.rows *= 2;
  const int64_t chunks = grouped ? live : cdiv(g.M, ch.rows);
  if (p.trans_b) {
    if (cdiv(g.N, 16) * chunks < kCUs) ch.cols = 4;
  } else {
    while (ch.cols > 16 && cdiv(g.N, ch.cols) * chunks < kCUs * 5 / 8) ch.cols /= 2;
    if (cdiv(g.N, ch.cols) * chunks < 2 * kCUs) ch.threads = 512;
  }
  const sg::host::TileCost c = {ch.rows, ch.cols, 0, 0, 0, 0, 0, 0};
  ch.workgroups = grid_tiles(g, c);
  return grid_fits(ch.workgroups, ch.threads) ? ch : none;
}

// Where a split, if there is room for one, is faster than so many rows over a B
// that the caches do not hold: see choose_rows.
bool many_rows(const Product& p) {
  const int64_t size = (int64_t)p.g.N * p.g.K;
  return p.g.mode == sg::kDense &&
         ((p.g.M > sg::kRowsMost && size > 1 << 23) ||
          (!p.trans_b && size > 1 << 24 && cdiv(p.g.N, 64) < kCUs * 5 / 8));
}

// Few columns over a long K leave the chip idle by rows, where a split product
// fills it.  Measured (us, rows / split; N x K):
//      B stored N x K   64 x 65536   64 x 16384   1024 x 8192
//      1 row             17.5 / 27.4    5.1 / 12.6    7.3 / 12.9
//      8 rows            40.4 / 27.4   10.8 / 13.3    9.7 / 12.9
//      B stored K x N   64 x 16384   256 x 4096   1024 x 8192   1024 x 1024
//      1 row             25.2 / 13.1    6.1 / 9.3    18.2 / 12.9    4.5 / 9.0
//      8 rows            58.2 / 13.3   13.0 / 9.8    28.8 / 12.9    5.5 / 9.2
bool rather_tiles(const Product& p, const RowsChoice& rows, const Choice& ch) {
  if (ch.v == nullptr) return false;
  if (many_rows(p))
    return ch.splits > 1 || (p.g.M > sg::kRowsMost && cdiv(p.g.N, 64) >= kCUs / 2 &&
                             (int64_t)p.g.N * p.g.K > 1 << 24);
  if (ch.splits == 1) return false;
  const int64_t K = p.g.K;
  return p.trans_b ? rows.workgroups < 64 && K * rows.rows > 196608
                   : rows.workgroups <= kCUs / 2 && K * (rows.rows + 2) > 12288;
}

// What one launch (or a split's two) of a product would be.
struct Step {
  RowsChoice rows;   // rows.rows > 0: by rows
  Choice tile;
};

Step decide(const Product& p, int64_t ws_bytes) {
  const RowsChoice rows = choose_rows(p);
  Step s = {{0, 0, 0, 0}, {nullptr, 1, 0, 0, 0.0}};
  // Only many rows, or a long K over few columns, ask what a split would be.
  if (rows.rows == 0 || many_rows(p) || (p.g.K > 1024 && rows.workgroups <= kCUs / 2))
    s.tile = choose(p, ws_bytes);
  if (rows.rows > 0 && !rather_tiles(p, rows, s.tile)) s.rows = rows;
  return s;
}

bool possible(const Step& s) { return s.rows.rows > 0 || s.tile.v != nullptr; }

int64_t step_bytes(const Product& p, const Step& s) {
  return s.rows.rows > 0 ? 0 : split_bytes(p.g, s.tile);
}

double step_seconds(const Product& p, const Step& s) {
  // By rows: reading B, and a launch.
  return s.rows.rows > 0 ? 4.0e-6 + 4.0 * p.g.N * p.g.K / 4.5e12 : s.tile.seconds;
}

// A dense product cut in two along M or N, each part a launch of its own: a
// grid a little over what the chip holds at once otherwise pays a whole round
// for its remainder, which alone takes a fitting kernel.
struct Cut {
  int64_t at;     // rows or columns of the first part; 0: not cut
  bool columns;
};

// Rows (columns) `from` on, `count` of them.
Product part_of(const Product& whole, bool columns, int64_t from, int64_t count) {
  Product p = whole;
  ProductArgs& g = p.g;
  if (columns) {
    g.B += p.trans_b ? from * g.ldb : from;
    g.C += from;
    if (g.bias) g.bias += from;
    if (g.residual) g.residual += from;
    if (g.preact) g.preact += from;
    g.N = (int)count;
  } else {
    g.A += p.trans_a ? from : from * g.lda;
    g.C += from * g.ldc;
    if (g.residual) g.residual += from * g.ldr;
    if (g.preact) g.preact += from * g.ldp;
    g.M = (int)count;
  }
  return p;
}

// The cut with the least estimated time, if it is 4% under the uncut product's:
// whole rounds of one of the three largest tiles, and the rest.  Not asked
// where the whole is short or near what the chip can do anyway.  Measured on
// MI355X (us, one launch / cut): 4097 x 4096 x 4096 1020 / 923, 8200 x 4096 x
// 4096 1992 / 1840, 16385 x 1024 x 1024 of an N x K weight 265 / 243.
Cut find_cut(const Product& p, const Step& whole, int64_t ws_bytes) {
  const ProductArgs& g = p.g;
  Cut best = {0, false};
  if (g.mode != sg::kDense || whole.rows.rows > 0 || whole.tile.v == nullptr) return best;
  const double t_whole = whole.tile.seconds;
  if (t_whole < 60e-6 || t_whole < 1.04 * 2.0 * g.M * g.N * g.K / 150e12) return best;
  double t_best = 0.96 * t_whole;
  const ProductVariant* table = variants(p.trans_a, p.trans_b);
  for (int i = 0; i < 3; ++i) {
    const sg::host::TileCost& c = table[i].cost;
    if (!variant_fits(p, table[i])) continue;
    const int64_t tm = cdiv(g.M, c.tile_m), tn = cdiv(g.N, c.tile_n);
    const int64_t round = (int64_t)kCUs * c.occ, full = tm * tn / round * round;
    for (int columns = 0; columns < 2; ++columns) {
      const int64_t tiles = full / (columns ? tm : tn);
      const int64_t at = tiles * (columns ? c.tile_n : c.tile_m), size = columns ? g.N : g.M;
      if (at <= 0 || at >= size) continue;
      const double t = estimate_grid(c, tiles * (columns ? tm : tn), g.K);
      if (t >= t_best) continue;
      const Product rest = part_of(p, columns, at, size - at);
      const double both = t + step_seconds(rest, decide(rest, ws_bytes)) + 2.0e-6;
      if (both < t_best) {
        t_best = both;
        best = {at, columns != 0};
      }
    }
  }
  return best;
}

int launch_step(Product& p, const Step& s, hipStream_t stream, void* ws) {
  ProductArgs& g = p.g;
  void* args[] = {&g};
  const int tile_m = s.rows.rows > 0 ? s.rows.rows : s.tile.v->cost.tile_m;
  const int tile_n = s.rows.rows > 0 ? s.rows.cols : s.tile.v->cost.tile_n;
  g.tiles_m = (int)cdiv(g.M, tile_m);
  g.tiles_n = (int)cdiv(g.N, tile_n);
  g.group_m = g.tiles_m < 8 ? g.tiles_m : 8;
  if (s.rows.rows > 0) {
    const hipError_t e = hipLaunchKernel(
        reinterpret_cast<const void*>(sg::rows_kernel(p.trans_b, s.rows.rows, s.rows.cols,
                                                          s.rows.threads, g.K >= 2048)),
        dim3((unsigned)s.rows.workgroups), dim3(s.rows.threads), args, 0, stream);
    return e == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
  }
  g.splits = s.tile.splits;
  g.k_split = s.tile.k_split;
  g.W = static_cast<float*>(ws);
  hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(s.tile.v->fn),
                                 dim3((unsigned)s.tile.workgroups), dim3(s.tile.v->cost.threads),
                                 args, 0, stream);
  if (e == hipSuccess && s.tile.splits > 1) {
    const int64_t rows = (int64_t)g.M * (g.mode == sg::kSumGroups ? g.groups : 1);
    e = hipLaunchKernel(reinterpret_cast<const void*>(sg::product_reduce_kernel),
                        dim3((unsigned)(rows * cdiv(g.N, sg::kProductReduceCols))), dim3(64), args,
                        0, stream);
  }
  return e == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

int run_product(Product& p, const int32_t* offsets, hipStream_t stream, void* ws,
                int64_t ws_bytes) {
  Product part[2] = {p, p};
  Step step[2] = {decide(p, ws_bytes), {}};
  if (!possible(step[0])) return SGEMM_ERR_UNSUPPORTED;
  const Cut cut = find_cut(p, step[0], ws_bytes);
  const int parts = cut.at > 0 ? 2 : 1;
  if (parts == 2) {
    part[0] = part_of(p, cut.columns, 0, cut.at);
    part[1] = part_of(p, cut.columns, cut.at, (cut.columns ? p.g.N : p.g.M) - cut.at);
    for (int i = 0; i < 2; ++i) {
      step[i] = decide(part[i], ws_bytes);
      if (!possible(step[i])) return SGEMM_ERR_UNSUPPORTED;
    }
  }
  // Everything is checked before the first launch.
  for (int i = 0; i < parts; ++i) {
    const Span w = {ws, step_bytes(part[i], step[i])};
    const Span off = {offsets, offsets ? (int64_t)(p.g.groups + 1) * 4 : 0};
    if (overlaps(w, p.a) || overlaps(w, p.b) || overlaps(w, p.c) || overlaps(w, p.bias) ||
        overlaps(w, p.res) || overlaps(w, p.pre) || overlaps(w, off))
      return SGEMM_ERR_INVALID_ARG;
  }
  for (int i = 0; i < parts; ++i) {
    const int st = launch_step(part[i], step[i], stream, ws);
    if (st != SGEMM_OK) return st;
  }
  return SGEMM_OK;
}

// A product with no operands, for the questions about plans.
Product shape_only(int mode, bool ta, bool tb, int64_t M, int64_t N, int64_t K, int64_t groups,
                   int64_t rows) {
  Product p;
  memset(&p, 0, sizeof(p));
  p.trans_a = ta;
  p.trans_b = tb;
  p.launch = M > 0 && N > 0 && groups > 0;
  p.g.M = (int)M;
  p.g.N = (int)N;
  p.g.K = (int)K;
  p.g.lda = (int)at_least_one(ta ? M : K);
  p.g.ldb = (int)at_least_one(tb ? K : N);
  p.g.ldc = (int)N;
  p.g.mode = mode;
  p.g.groups = (int)groups;
  p.g.rows = (int)rows;
  return p;
}

bool sizes_ok(int64_t a, int64_t b, int64_t c) {
  return a >= 0 && b >= 0 && c >= 0 && a <= kMaxDim && b <= kMaxDim && c <= kMaxDim;
}

int64_t plan_workspace(const Product& p) {
  if (!p.launch) return 0;
  const Step s = decide(p, INT64_MAX);
  const Cut cut = find_cut(p, s, INT64_MAX);
  if (cut.at == 0) return step_bytes(p, s);
  const Product a = part_of(p, cut.columns, 0, cut.at);
  const Product b = part_of(p, cut.columns, cut.at, (cut.columns ? p.g.N : p.g.M) - cut.at);
  const int64_t x = step_bytes(a, decide(a, INT64_MAX)), y = step_bytes(b, decide(b, INT64_MAX));
  return x > y ? x : y;
}

int act_lanes(int64_t N) {
  int lpr = 64;
  while (lpr > 1 && 2 * N <= 4 * lpr) lpr /= 2;
  return lpr;
}

// Up to so many workgroups of 16 columns add the spans' sums; where there would be
// more, of 1024 threads with little to do, they take 128 (us, both passes, by 16 and
// by 128: 4096 x 4096 of 128 groups 82 / 45, 8190 x 1500 of 16 39 / 35, 256 x 1024 of
// 8 8.3 / 8.0, 65536 x 128 of one 23 / 33).
constexpr int64_t kSumNarrow = 1024;

// How the activation pass cuts the rows: into spans of so many, each group's
// counted from its first row, and how many of them there can be.
struct ActSpans {
  int64_t rows, most;
};

// Spans enough for four workgroups a CU, of at least four rounds of rows.  The
// lengths of the groups are not known here: `groups` ends add as many spans.
// Sums of several spans take a second launch: over groups with no more than 32
// rounds in all a span each, without it (us, both ways: 128 rows of 8 groups, N =
// 2048, 5.3 / 9.9; 256 rows, past it, 8.1, and 7.5 with all of them in one group,
// where a span each took 24).
ActSpans act_spans(int64_t M, int64_t N, int64_t groups, bool grouped, bool sums) {
  const int lpr = act_lanes(N), beside = 64 / lpr * sg::kActWaves;
  int64_t s = cdiv(4 * kCUs, cdiv(N, 4 * lpr));
  const int64_t most = cdiv(M, 4 * beside);
  if (s > most) s = most;
  if (s < 1 || (grouped && sums && M <= 32 * beside)) s = 1;
  const int64_t rows = at_least_one(cdiv(M, s));
  return {rows, grouped ? M / rows + groups : at_least_one(cdiv(M, rows))};
}

int64_t act_workspace(int64_t M, int64_t N, int64_t groups, bool grouped) {
  if (M <= 0 || N <= 0 || groups <= 0 || M > kMaxDim || N > kMaxDim || groups > sg::kMaxGroups)
    return 0;
  const ActSpans s = act_spans(M, N, groups, grouped, true);
  return M > s.rows ? s.most * N * 4 : 0;
}

int act_backward(int64_t M, int64_t N, int64_t groups, const int32_t* offsets, bool grouped,
                 const float* dC, int64_t lddc, const float* Z, int64_t ldz, int act, float* dZ,
                 int64_t lddz, float* dbias, int64_t lddb, hipStream_t stream, void* ws,
                 int64_t ws_bytes) {
  if (M < 0 || N < 0 || groups < 0 || act < SGEMM_ACT_NONE || act > SGEMM_ACT_SILU)
    return SGEMM_ERR_INVALID_ARG;
  if (ws_bytes < 0 || (ws_bytes > 0 && ws == nullptr) || ((uintptr_t)ws & 3u))
    return SGEMM_ERR_INVALID_ARG;
  const int64_t n1 = at_least_one(N);
  if (act == SGEMM_ACT_NONE) Z = nullptr;
  if (lddc < n1 || (act != SGEMM_ACT_NONE && ldz < n1) || (dZ && lddz < n1) ||
      (grouped && dbias && lddb < n1))
    return SGEMM_ERR_INVALID_ARG;
  if (groups > sg::kMaxGroups) return SGEMM_ERR_UNSUPPORTED;
  if (N == 0 || groups == 0 || (!dZ && !dbias) || (M == 0 && !dbias)) return SGEMM_OK;
  const Span c = {dC, span_bytes(M, N, lddc)};
  const Span z = {Z, act != SGEMM_ACT_NONE ? span_bytes(M, N, ldz) : 0};
  const Span d = {dZ, dZ ? span_bytes(M, N, lddz) : 0};
  const Span b = {dbias, !dbias ? 0 : grouped ? groups_bytes(groups, lddb, floats(N)) : floats(N)};
  const Span off = {offsets, grouped ? (groups + 1) * 4 : 0};
  const Span all[] = {c, z, d, b, off};
  const int st = check_spans(all, 5);
  if (st != SGEMM_OK) return st;
  if (M > kMaxDim || N > kMaxDim) return SGEMM_ERR_UNSUPPORTED;
  const bool on_c = dZ == dC && lddz == lddc, on_z = Z && dZ == Z && lddz == ldz;
  if ((!on_c && overlaps(d, c)) || (!on_z && overlaps(d, z)) || overlaps(b, c) ||
      overlaps(b, z) || overlaps(b, d) || overlaps(off, d) || overlaps(off, b))
    return SGEMM_ERR_INVALID_ARG;

  ActBackwardArgs a;
  a.dC = dC;
  a.Z = Z;
  a.dZ = dZ;
  a.dbias = dbias;
  a.lddc = lddc;
  a.ldz = ldz;
  a.lddz = lddz;
  a.lddb = grouped ? lddb : 0;
  a.offsets = grouped ? offsets : nullptr;
  a.M = (int)M;
  a.N = (int)N;
  a.groups = (int)groups;
  a.lpr = act_lanes(N);
  a.blocks_n = (int)cdiv(N, 4 * a.lpr);
  const ActSpans spans = act_spans(M, N, groups, grouped, dbias != nullptr);
  a.span = (int)spans.rows;
  a.spans = (int)spans.most;
  // Room for the sums, where a group can have several spans.
  const int64_t need = dbias && M > spans.rows ? spans.most * N * 4 : 0;
  const Span w = {ws, ws_bytes < need ? ws_bytes : need};
  if (overlaps(w, c) || overlaps(w, z) || overlaps(w, d) || overlaps(w, b) || overlaps(w, off))
    return SGEMM_ERR_INVALID_ARG;
  const bool room = need > 0 && ws_bytes >= need;
  a.W = room ? static_cast<float*>(ws) : nullptr;
  const int64_t wgs = a.blocks_n * spans.most;
  if (!grid_fits(wgs, 64 * sg::kActWaves)) return SGEMM_ERR_UNSUPPORTED;
  void* kargs[] = {&a};
  typedef void (*ActFn)(ActBackwardArgs);
  static const ActFn table[] = {
      sg::act_backward_kernel<SGEMM_ACT_NONE>, sg::act_backward_kernel<SGEMM_ACT_RELU>,
      sg::act_backward_kernel<SGEMM_ACT_GELU>, sg::act_backward_kernel<SGEMM_ACT_GELU_TANH>,
      sg::act_backward_kernel<SGEMM_ACT_SILU>};
  hipError_t e = hipSuccess;
  // Nothing to do where act_sum_kernel does everything.
  if (dZ || room || need == 0 || grouped)
    e = hipLaunchKernel(reinterpret_cast<const void*>(table[act]), dim3((unsigned)wgs),
                        dim3(64 * sg::kActWaves), kargs, 0, stream);
  if (e != hipSuccess || need == 0) return e == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
  // Groups that can have several spans.
  const int64_t several = groups < (M - 1) / spans.rows ? groups : (M - 1) / spans.rows;
  int cols = 16, threads = 1024;
  const void* fn = reinterpret_cast<const void*>(sg::column_sum_kernel<16>);
  if (room && cdiv(N, 16) * several > kSumNarrow) {
    cols = 128;
    threads = sg::kSumThreads<128>;
    fn = reinterpret_cast<const void*>(sg::column_sum_kernel<128>);
  } else if (!room) {
    cols = a.lpr < 4 ? 4 * a.lpr : 16;
    if (dZ) {
      a.dC = dZ;
      a.lddc = lddz;
    }
    static const ActFn sums[] = {
        sg::act_sum_kernel<SGEMM_ACT_NONE>, sg::act_sum_kernel<SGEMM_ACT_RELU>,
        sg::act_sum_kernel<SGEMM_ACT_GELU>, sg::act_sum_kernel<SGEMM_ACT_GELU_TANH>,
        sg::act_sum_kernel<SGEMM_ACT_SILU>};
    fn = reinterpret_cast<const void*>(sums[dZ ? SGEMM_ACT_NONE : act]);
  }
  e = hipLaunchKernel(fn, dim3((unsigned)(cdiv(N, cols) * several)), dim3(threads), kargs, 0,
                      stream);
  return e == hipSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int sgemm_linear(int trans_a, int trans_b, int64_t M, int64_t N, int64_t K, const float* A,
                 int64_t lda, const float* B, int64_t ldb, float* C, int64_t ldc,
                 const sgemm_epilogue* epilogue, hipStream_t stream, void* workspace,
                 int64_t workspace_bytes) {
  Product p;
  const int st = check_product(sg::kDense, trans_a, trans_b, M, N, K, 0, nullptr, 0, A, lda, B,
                               ldb, 0, C, ldc, 0, epilogue, workspace, workspace_bytes, p);
  if (st != SGEMM_OK || !p.launch) return st;
  return run_product(p, p.g.offsets, stream, workspace, workspace_bytes);
}

int64_t sgemm_linear_workspace_bytes(int trans_a, int trans_b, int64_t M, int64_t N, int64_t K) {
  if (!sizes_ok(M, N, K) || ((trans_a | trans_b) & ~1)) return 0;
  return plan_workspace(shape_only(sg::kDense, trans_a, trans_b, M, N, K, 1, 0));
}

int sgemm_linear_plan_query(int trans_a, int trans_b, int64_t M, int64_t N, int64_t K,
                            int64_t workspace_bytes, sgemm_plan* plan) {
  if (plan == nullptr || workspace_bytes < 0 || M < 0 || N < 0 || K < 0 ||
      ((trans_a | trans_b) & ~1))
    return SGEMM_ERR_INVALID_ARG;
  if (!sizes_ok(M, N, K)) return SGEMM_ERR_UNSUPPORTED;
  memset(plan, 0, sizeof(*plan));
  plan->splits = 1;
  const Product p = shape_only(sg::kDense, trans_a, trans_b, M, N, K, 1, 0);
  if (!p.launch) return SGEMM_OK;
  const Step whole = decide(p, workspace_bytes);
  if (!possible(whole)) return SGEMM_ERR_UNSUPPORTED;
  // Of a product cut in two, the first part, and the workspace of both.
  const Cut cut = find_cut(p, whole, workspace_bytes);
  const Product first = cut.at > 0 ? part_of(p, cut.columns, 0, cut.at) : p;
  const Step s = cut.at > 0 ? decide(first, workspace_bytes) : whole;
  plan->vec_a = plan->vec_b = 1;
  plan->workspace_bytes = step_bytes(first, s);
  char rest[24] = "";
  if (cut.at > 0) {
    const Product b = part_of(p, cut.columns, cut.at, (cut.columns ? N : M) - cut.at);
    const int64_t more = step_bytes(b, decide(b, workspace_bytes));
    if (more > plan->workspace_bytes) plan->workspace_bytes = more;
    snprintf(rest, sizeof(rest), "+%d%s", cut.columns ? b.g.N : b.g.M, cut.columns ? "cols" : "rows");
  }
  if (s.rows.rows > 0) {
    plan->algo = SGEMM_ALGO_FMA;
    plan->tile_m = s.rows.rows;
    plan->tile_n = s.rows.cols;
    plan->threads = s.rows.threads;
    plan->workgroups = s.rows.workgroups;
    snprintf(plan->kernel, sizeof(plan->kernel), "rows_%s_%dx%d%s", trans_b ? "fast" : "slow",
             s.rows.rows, s.rows.cols, rest);
    return SGEMM_OK;
  }
  const sg::host::TileCost& c = s.tile.v->cost;
  plan->algo = SGEMM_ALGO_MFMA_DIRECT;
  plan->tile_m = c.tile_m;
  plan->tile_n = c.tile_n;
  plan->tile_k = c.tile_k;
  plan->threads = c.threads;
  plan->workgroups = s.tile.workgroups;
  plan->lds_bytes = s.tile.v->lds_bytes;
  plan->wg_per_cu = c.occ;
  plan->splits = s.tile.splits;
  snprintf(plan->kernel, sizeof(plan->kernel), "product_%c%c_%s%s", trans_a ? 's' : 'f',
           trans_b ? 'f' : 's', s.tile.v->name, rest);
  return SGEMM_OK;
}

int sgemm_act_backward(int64_t M, int64_t N, const float* dC, int64_t lddc, const float* preact,
                       int64_t ldp, int act, float* dZ, int64_t lddz, float* dbias,
                       hipStream_t stream, void* workspace, int64_t workspace_bytes) {
  return act_backward(M, N, 1, nullptr, false, dC, lddc, preact, ldp, act, dZ, lddz, dbias, 0,
                      stream, workspace, workspace_bytes);
}

int64_t sgemm_act_backward_workspace_bytes(int64_t M, int64_t N) {
  return act_workspace(M, N, 1, false);
}

int sgemm_grouped(int trans_b, int64_t M, int64_t N, int64_t K, int64_t groups,
                  const int32_t* offsets, const float* A, int64_t lda, const float* B,
                  int64_t ldb, int64_t stride_b, float* C, int64_t ldc,
                  const sgemm_epilogue* epilogue, hipStream_t stream, void* workspace,
                  int64_t workspace_bytes) {
  Product p;
  const int st = check_product(sg::kRowGroups, 0, trans_b, M, N, K, groups, offsets, M, A, lda, B,
                               ldb, stride_b, C, ldc, 0, epilogue, workspace, workspace_bytes, p);
  if (st != SGEMM_OK || !p.launch) return st;
  return run_product(p, p.g.offsets, stream, workspace, workspace_bytes);
}

int64_t sgemm_grouped_workspace_bytes(int trans_b, int64_t M, int64_t N, int64_t K,
                                      int64_t groups) {
  if (!sizes_ok(M, N, K) || groups < 0 || groups > sg::kMaxGroups || (trans_b & ~1)) return 0;
  return plan_workspace(shape_only(sg::kRowGroups, false, trans_b, M, N, K, groups, M));
}

// dB_g of K x N is a product of K x rows (A transposed) and rows x N; its
// transpose one of N x rows and rows x K.
int sgemm_grouped_wgrad(int trans_b, int64_t M, int64_t N, int64_t K, int64_t groups,
                        const int32_t* offsets, const float* A, int64_t lda, const float* dZ,
                        int64_t lddz, float* dB, int64_t lddb, int64_t stride_db,
                        hipStream_t stream, void* workspace, int64_t workspace_bytes) {
  if (trans_b & ~1) return SGEMM_ERR_INVALID_ARG;
  Product p;
  const int st = check_product(sg::kSumGroups, 1, 0, trans_b ? N : K, trans_b ? K : N, M, groups,
                               offsets, M, trans_b ? dZ : A, trans_b ? lddz : lda,
                               trans_b ? A : dZ, trans_b ? lda : lddz, 0, dB, lddb, stride_db,
                               nullptr, workspace, workspace_bytes, p);
  if (st != SGEMM_OK || !p.launch) return st;
  return run_product(p, p.g.offsets, stream, workspace, workspace_bytes);
}

int64_t sgemm_grouped_wgrad_workspace_bytes(int trans_b, int64_t M, int64_t N, int64_t K,
                                            int64_t groups) {
  if (!sizes_ok(M, N, K) || groups < 0 || groups > sg::kMaxGroups || (trans_b & ~1)) return 0;
  return plan_workspace(shape_only(sg::kSumGroups, true, false, trans_b ? N : K, trans_b ? K : N,
                                   M, groups, M));
}

int sgemm_grouped_act_backward(int64_t M, int64_t N, int64_t groups, const int32_t* offsets,
                               const float* dC, int64_t lddc, const float* preact, int64_t ldp,
                               int act, float* dZ, int64_t lddz, float* dbias, int64_t lddbias,
                               hipStream_t stream, void* workspace, int64_t workspace_bytes) {
  return act_backward(M, N, groups, offsets, true, dC, lddc, preact, ldp, act, dZ, lddz, dbias,
                      lddbias, stream, workspace, workspace_bytes);
}

int64_t sgemm_grouped_act_backward_workspace_bytes(int64_t M, int64_t N, int64_t groups) {
  return act_workspace(M, N, groups, true);
}

}  // extern "C"
