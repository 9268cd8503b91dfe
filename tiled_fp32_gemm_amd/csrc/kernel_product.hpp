// kernel_product.hpp -- FP32 matrix-core products with either operand
// transposed, an epilogue, and groups.
//
// The main loop is that of kernel_mfma_direct.hpp: slabs of BK values of k go
// from global memory straight into LDS (STAGES of them, all but one in flight),
// the waves read their fragments one 8-deep chunk ahead of the 32x32x2 matrix
// instructions, and the slab barrier sits before a slab's last chunk.  Bound by
// the matrix pipe on full grids; measured on MI355X at 4096^3 (137.4 GFLOP,
// 256 x 256 tiles): 914 us with A k fast and B k slow, 918 both fast, 916 both
// slow, 916 the other way round, where sgemm takes 913 (150.5 TFLOP/s).  What is
// new here:
//
// Operand layouts.  An operand is stored either with k running along its rows
// (A as M x K, B as N x K: "k fast") or with k from row to row (A as K x M, B
// as K x N: "k slow"), and there are two LDS layouts to match, both permutations
// of 16-byte units that keep every direct load lane-linear and every fragment
// read conflict-free on 64 banks of 4 bytes (R: the tile's extent, CPR = BK/4):
//   k fast   unit(r, c) = CPR r + (c xor r / (16 / CPR) mod CPR): a lane's four
//            values of k come in one 128-bit read, 16 rows read all 64 banks,
//            and neighbouring lanes of a direct load fetch one row's cache line.
//            The 256 x 256 tile, which has no register left for the xor's four
//            addresses and loads little for what it computes, has
//            unit(r, c) = 16 CPR (r / 16) + 16 c + r % 16, whose lanes fetch 16
//            bytes of 16 rows.  With that in the smaller tiles the loads bound
//            them, at 8.4 to 9 TB/s over the chip: 64 x 11008 x 4096 of an N x K
//            weight 78.7 -> 61.5 us, 128 x 4096 x 4096 52.5 -> 46.6, 64 x 64 tiles
//            at 4096^3 132 -> 143 TFLOP/s;
//   k slow   unit(k, q) = (k R/4 + q) xor (k & 8): lanes 0-31 read row 16 s + p
//            and lanes 32-63 row 16 s + 8 + p; the xor puts the two on
//            different halves of the banks (within a row when R >= 64, on the
//            neighbouring row when R = 32).  With two 32-blocks per wave, block
//            j takes the wave's rows or columns 2 i + j, so that a lane's two
//            words of a k step are adjacent: one 64-bit read.
// The instruction takes k = lane / 32 from both operands alike, so either
// layout can feed either side.  k past the end reads zeros: beyond the resource
// when k is slow, zeroed in LDS after the load when it is fast.
//
// Groups (product_args.hpp).  kRowGroups: the workgroups share out the tiles of
// all groups' row ranges, which only the device knows; each wave scans the
// offsets for its own tile, and workgroups past the last tile leave at once.
// kSumGroups: every group has the same tiles and a k range of its own.
//
// Epilogue.  The accumulators go through LDS, 32 rows of a wave at a time (each
// wave in its own part, no barrier), so that bias, activation and residual are
// applied four columns a lane in a short loop and every global access is 16
// bytes a lane along a row.  The residual's loads are issued before the
// activation runs, for small wave tiles before the main loop.  At 4096^3 a bias
// costs 6 us, GELU 10, a residual 12, all of them and the stored
// pre-activation 27 (192 MiB more to move).  Split K (splits > 1) stores the
// partial sums instead; kernel_product_reduce.hpp adds them and applies the
// epilogue.
#pragma once

#include <type_traits>

#include "activation.hpp"
#include "product_args.hpp"
#include "rows.hpp"

namespace sg {

template <int BM, int BN, int WM, int WN, int BK_, int KS_, int STAGES_>
struct ProductCfg {
  static constexpr int BK = BK_, KS = KS_, STAGES = STAGES_;
  static constexpr int CPR = BK / 4;
  static constexpr int SUB_G = BK / 16 / KS;   // 16-deep sub-slabs per wave group
  static constexpr int WAVES_N = BN / WN;
  static constexpr int SPATIAL = (BM / WM) * (BN / WN);
  static constexpr int NT = 64 * SPATIAL * KS;
  static constexpr int TA = WM / 32, TB = WN / 32;
  static constexpr int A_STAGE = BM * BK, B_STAGE = BK * BN;   // floats
  static constexpr int STAGE_FLOATS = STAGES * (A_STAGE + B_STAGE);
  static constexpr int RED_FLOATS = (KS - 1) * BM * BN;
  static constexpr int OUT_FLOATS = SPATIAL * 32 * WN;
  static constexpr bool LINES = BM * BN < 256 * 256;   // the k-fast layout
  static constexpr int max3(int a, int b, int c) {
    return a > b ? (a > c ? a : c) : (b > c ? b : c);
  }
  static constexpr int LDS_FLOATS = max3(STAGE_FLOATS, RED_FLOATS, OUT_FLOATS);
  static constexpr int A_SLOTS = BM * BK / 4 / NT, B_SLOTS = BK * BN / 4 / NT;
  static constexpr int LOADS = A_SLOTS + B_SLOTS;
  static_assert(A_SLOTS * NT * 4 == BM * BK && B_SLOTS * NT * 4 == BK * BN, "whole loads");
  static_assert(BM % 32 == 0 && BN % 32 == 0 && BK % 16 == 0 && TA <= 2 && TB <= 2, "tile");
  static_assert(SUB_G * KS * 16 == BK, "whole sub-slabs per wave group");
};

// s_waitcnt immediates for this wave's vector-memory operations and for its LDS
// accesses (the other counts at their maxima).
template <int n>   // at most n vector-memory operations left
constexpr int kWaitLoads = (n & 0xF) | (0x7 << 4) | (0xF << 8) | ((n >> 4) << 14);
constexpr int kWaitLds = 0xF | (0x7 << 4) | (0x3 << 14);

// What a k-fast row's k groups are xor-ed with: sixteen consecutive rows take the
// sixteen 16-byte units of 64 banks for every k group.
template <int CPR>
__device__ __forceinline__ int fast_swizzle(int r) {
  static_assert(CPR == 4 || CPR == 8 || CPR == 16, "16, 32 or 64 values of k a slab");
  return (r / (16 / CPR)) & (CPR - 1);
}

// Where one operand's unit u of a slab stage comes from: for k fast the row
// (of the tile) and k group, for k slow the k and the 4-float group.
template <bool FAST, int R, int CPR, bool LINES>
__device__ __forceinline__ void unit_source(int u, int& r, int& k) {
  if constexpr (FAST && LINES) {
    r = u / CPR;
    k = 4 * ((u % CPR) ^ fast_swizzle<CPR>(r));
  } else if constexpr (FAST) {
    r = (u / (16 * CPR)) * 16 + (u & 15);
    k = 4 * ((u >> 4) % CPR);
  } else {
    const int v = u ^ (((u / (R / 4)) & 8) ? 8 : 0);
    k = v / (R / 4);
    r = 4 * (v % (R / 4));
  }
}

// A group's tile for workgroup w of a kRowGroups grid.
struct RowTile {
  int group, first, end;   // rows first .. end-1 of the group's range from its tile on
  int tm, tn, split;
};

// Workgroup ids are handed to the 8 XCDs round-robin: renumbered so that the
// ids of one XCD are consecutive.
__device__ __forceinline__ int xcd_order(int w, int n) {
  const int q = n >> 3, rem = n & 7, xcd = w & 7;
  return xcd * q + (xcd < rem ? xcd : rem) + (w >> 3);
}

// Consecutive ids walk a group of rows of tiles column by column.
__device__ __forceinline__ void tile_order(int L, int tiles_m, int tiles_n, int group_m, int& tm,
                                           int& tn) {
  const int per = group_m * tiles_n;
  const int grp = L / per;
  const int rows = min(tiles_m - grp * group_m, group_m);
  const int in = L - grp * per;
  tm = grp * group_m + in % rows;
  tn = in / rows;
}

// False: no tile for this workgroup.  The groups' whole tiles come first, in
// group order, then their partial last ones, which are shorter work: the
// launch ends with them, and each XCD has its share of both.  Tiles of 128 rows
// and more are sorted by length there: 16384 rows of sixteen uneven groups, N =
// 4096, K = 1024, 256-row tiles 1179 -> 1024 us, 128-row tiles 1070 -> 1020 us
// (64-row tiles lose by it, as neighbours part: 88 -> 95 us for 4096 rows of
// eight groups, N = K = 1024).  Every wave does this for itself, 64 groups at a
// time, and almost always has all of them at once.
template <int BM>
__device__ __forceinline__ bool row_group_tile(const ProductArgs& g, int lane, RowTile& t) {
  int b = 0, e = 0, whole = 0, upto = 0;
  bool part = false;   // looking for partial tiles
  auto scan = [&](int e0) {
    b = e = 0;
    if (e0 + lane < g.groups) group_range(g.offsets, e0 + lane, g.rows, b, e);
    whole = (e - b) / BM;
    upto = scan64(part ? ((e - b) % BM != 0 ? 1 : 0) : whole);
  };
  auto count = [&]() {
    scan(0);
    int n = __builtin_amdgcn_readlane(upto, 63);
    if (g.groups > 64) {
      for (int e0 = 64; e0 < g.groups; e0 += 64) {
        scan(e0);
        n += __builtin_amdgcn_readlane(upto, 63);
      }
      scan(0);
    }
    return n * g.tiles_n;
  };
  int w = (int)blockIdx.x;
  int total = count();
  if (w >= total * g.splits) {
    w -= total * g.splits;
    part = true;
    total = count();
    if (w >= total * g.splits) return false;
  }
  // Large partial tiles go out longest first and to the XCDs in turn, so that
  // the launch does not end on a long one.
  const bool ranked = BM >= 128 && part && g.groups <= 64;
  int L = ranked ? w : xcd_order(w, total * g.splits);
  t.split = L / total;
  L -= t.split * total;
  const int row_tile = L / g.tiles_n;   // of all groups' row tiles
  if (ranked) {
    const int rem = (e - b) % BM;
    int rank = 0;   // groups with a longer partial tile
    for (int j = 0; j < g.groups; ++j) {
      const int other = __builtin_amdgcn_readlane(rem, j);
      rank += other > rem || (other == rem && j < lane) ? 1 : 0;
    }
    const uint64_t hit = __ballot(rem > 0 && rank == row_tile);
    if (hit == 0) return false;
    const int at = __ffsll((unsigned long long)hit) - 1;
    t.group = at;
    t.first = __builtin_amdgcn_readlane(b, at);
    t.end = __builtin_amdgcn_readlane(e, at);
    t.tm = __builtin_amdgcn_readlane(whole, at);
    t.tn = L - row_tile * g.tiles_n;
    return t.tn >= 0 && t.tn < g.tiles_n && t.first + t.tm * BM < t.end;
  }
  int before = 0;
  for (int e0 = 0;;) {
    const uint64_t past = __ballot(before + upto > row_tile);
    if (past != 0) {
      const int at = __ffsll((unsigned long long)past) - 1;
      const int rows = __builtin_amdgcn_readlane(whole, at);
      const int tiles_m = part ? 1 : rows;
      L -= (before + __builtin_amdgcn_readlane(upto, at) - tiles_m) * g.tiles_n;
      t.group = e0 + at;
      t.first = __builtin_amdgcn_readlane(b, at);
      t.end = __builtin_amdgcn_readlane(e, at);
      tile_order(L, tiles_m, g.tiles_n, min(tiles_m, 8), t.tm, t.tn);
      // Offsets that fall could make the counts above overflow.
      const bool good = t.tm >= 0 && t.tm < tiles_m && t.tn >= 0 && t.tn < g.tiles_n;
      if (part) t.tm = rows;
      return good && t.first + t.tm * BM < t.end;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
    e0 += 64;
    if (e0 >= g.groups) return false;
    scan(e0);
  }
}

// The group in place `place` of a kSumGroups grid and its range.  Up to sixteen
// groups go longest first, so that the launch ends on short ones: 16384 rows of
// sixteen, 1024 x 4096 outputs each, 1034 -> 983 us, 8190 rows, 777 x 1500, 178 ->
// 173 us.  With more groups the sorting, which every wave does, costs more than
// it gives (forty: 183 -> 196 us).
__device__ __forceinline__ void sum_group(const ProductArgs& g, int place, int lane, int& group,
                                          int& begin, int& end) {
  group = place;
  if (g.groups <= 16) {
    int b = 0, e = 0, rank = 0;   // rank: groups before this lane's
    if (lane < g.groups) group_range(g.offsets, lane, g.rows, b, e);
    for (int j = 0; j < g.groups; ++j) {
      const int other = __builtin_amdgcn_readlane(e - b, j);
      rank += other > e - b || (other == e - b && j < lane) ? 1 : 0;
    }
    const uint64_t hit = __ballot(lane < g.groups && rank == place);
    group = __ffsll((unsigned long long)hit) - 1;   // the ranks are 0 .. groups-1
    begin = __builtin_amdgcn_readlane(b, group);
    end = __builtin_amdgcn_readlane(e, group);
  } else {
    group_range(g.offsets, group, g.rows, begin, end);
  }
}

// AFAST: A is M x K.  BFAST: B is N x K.
template <int BM, int BN, int WM, int WN, int BK_, int KS_, int STAGES_, bool AFAST, bool BFAST>
__global__ void __launch_bounds__(64 * (BM / WM) * (BN / WN) * KS_)
product_kernel(ProductArgs g) {
  using Cfg = ProductCfg<BM, BN, WM, WN, BK_, KS_, STAGES_>;
  constexpr int S = Cfg::STAGES;
  constexpr int BK = Cfg::BK, NT = Cfg::NT, TA = Cfg::TA, TB = Cfg::TB, CPR = Cfg::CPR;
  constexpr int KS = Cfg::KS, SUB_G = Cfg::SUB_G;
  __shared__ __attribute__((aligned(16))) float lds[Cfg::LDS_FLOATS];
  float* const As = lds;                      // [S][A_STAGE]
  float* const Bs = lds + S * Cfg::A_STAGE;   // [S][B_STAGE]

  const int tid = (int)threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = KS == 1 ? 0 : wave / Cfg::SPATIAL;
  const int sw = KS == 1 ? wave : wave % Cfg::SPATIAL;
  const int wm0 = (sw / Cfg::WAVES_N) * WM;
  const int wn0 = (sw % Cfg::WAVES_N) * WN;
  const int li = lane & 31, lh = lane >> 5;

  // This workgroup's product: m_left x n_left outputs from (row0, n0) of C on,
  // over K values of k from kb on.
  int row0, n0, m_left, kb, K, group = 0, split;
  if (g.mode == kRowGroups) {
    RowTile t;
    if (!row_group_tile<BM>(g, lane, t)) return;
    group = t.group;
    split = t.split;
    row0 = t.first + t.tm * BM;
    m_left = t.end - row0;
    n0 = t.tn * BN;
    kb = split * g.k_split;
    K = g.splits > 1 ? min(g.k_split, g.K - kb) : g.K;
  } else {
    // Summed groups differ in length: the XCDs share each group's tiles, rather
    // than take whole groups.
    const int tiles = g.tiles_m * g.tiles_n;
    const int per_group = g.mode == kSumGroups ? tiles * g.splits : (int)gridDim.x;
    group = (int)blockIdx.x / per_group;
    const int L = xcd_order((int)blockIdx.x - group * per_group, per_group);
    split = L / tiles;
    int tm, tn;
    tile_order(L - split * tiles, g.tiles_m, g.tiles_n, g.group_m, tm, tn);
    row0 = tm * BM;
    m_left = g.M - row0;
    n0 = tn * BN;
    int first = 0, end = g.K, per = g.k_split;
    if (g.mode == kSumGroups) {
      sum_group(g, group, lane, group, first, end);
      // Whole slabs for every split, the last ones shorter or empty.
      per = ((end - first + g.splits - 1) / g.splits + BK - 1) / BK * BK;
    }
    kb = first;
    K = end - first;
    if (g.splits > 1) {
      const int skip = (int)min((int64_t)split * per, (int64_t)K);
      kb += skip;
      K = min(K - skip, per);
    }
  }
  // The same for every lane, which the compiler cannot tell of loaded values.
  row0 = __builtin_amdgcn_readfirstlane(row0);
  n0 = __builtin_amdgcn_readfirstlane(n0);
  m_left = __builtin_amdgcn_readfirstlane(m_left);
  kb = __builtin_amdgcn_readfirstlane(kb);
  K = __builtin_amdgcn_readfirstlane(K);
  group = __builtin_amdgcn_readfirstlane(group);
  split = __builtin_amdgcn_readfirstlane(split);
  const int n_left = g.N - n0;

  // The lane's four columns and rows in the epilogue: LPR lanes take a row's
  // 16-byte groups, so IT rounds cover 32 rows.  Small wave tiles have registers
  // to spare and load the bias and the residual now, under the main loop; the
  // large ones do after it.
  constexpr int LPR = WN / 4, RPI = 64 / LPR, IT = 32 / RPI;
  constexpr bool kEarly = TA * TB == 1;
  const bool partial = g.splits > 1;
  const bool has_bias = !partial && g.bias != nullptr;
  const float* res = partial || !g.residual ? nullptr : g.residual + (int64_t)row0 * g.ldr + n0;
  f32x4 bias = {0.0f, 0.0f, 0.0f, 0.0f}, add[IT];
  auto load_bias = [&](int ln) {
    const int cols = n_left - wn0 - 4 * (ln % LPR);
    if (has_bias && cols > 0)
      bias = load_upto(g.bias + group * g.ld_bias + n0 + wn0 + 4 * (ln % LPR), cols);
  };
  // Row q of block i of the wave tile, from the tile's first row.
  constexpr bool kPairA = !AFAST && TA == 2, kPairB = !BFAST && TB == 2;
  auto row_of = [&](int i, int q) { return wm0 + (kPairA ? 2 * q + i : 32 * i + q); };
  auto load_residual = [&](int i, int ln) {
    const int col = wn0 + 4 * (ln % LPR), cols = n_left - col;
    if (!res) return;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int row = row_of(i, it * RPI + ln / LPR);
      if (row < m_left && cols > 0)
        add[it] = load_upto(res + (uint32_t)row * (uint32_t)g.ldr + (uint32_t)col, cols);
    }
  };
  if (kEarly && grp == 0) {
    load_bias(lane);
    load_residual(0, lane);
  }

  // The tile's corner of each operand, and the bytes of it from there to the
  // last element this tile reads (one tile's rows when k is fast).
  const float* At = AFAST ? g.A + (int64_t)row0 * g.lda + kb : g.A + (int64_t)kb * g.lda + row0;
  const float* Bt = (g.mode == kRowGroups ? g.B + group * g.stride_b : g.B) +
                    (BFAST ? (int64_t)n0 * g.ldb + kb : (int64_t)kb * g.ldb + n0);
  const int64_t a_rem = 4 * (AFAST ? (int64_t)(min(m_left, BM) - 1) * g.lda + K
                                   : (int64_t)(K - 1) * g.lda + m_left);
  const int64_t b_rem = 4 * (BFAST ? (int64_t)(min(n_left, BN) - 1) * g.ldb + K
                                   : (int64_t)(K - 1) * g.ldb + n_left);
  const uint32_t a_cap = (uint32_t)a_rem, b_cap = (uint32_t)b_rem;   // k fast only

  // The offset of the group each lane loads in every slab.
  auto offset = [&](auto fast, int r, int k, int left, int ld) -> uint32_t {
    if constexpr (decltype(fast)::value)
      return r < left ? ((uint32_t)r * (uint32_t)ld + (uint32_t)k) * 4u : kOob;
    else   // with K < BK the rows past K may lie 2^31 bytes away
      return r < left && k < K ? ((uint32_t)k * (uint32_t)ld + (uint32_t)r) * 4u : kOob;
  };
  using AFastT = std::integral_constant<bool, AFAST>;
  using BFastT = std::integral_constant<bool, BFAST>;
  uint32_t a_off[Cfg::A_SLOTS], b_off[Cfg::B_SLOTS];
#pragma unroll
  for (int s = 0; s < Cfg::A_SLOTS; ++s) {
    int r, k;
    unit_source<AFAST, BM, CPR, Cfg::LINES>(s * NT + 64 * wave + lane, r, k);
    a_off[s] = offset(AFastT(), r, k, m_left, g.lda);
  }
#pragma unroll
  for (int s = 0; s < Cfg::B_SLOTS; ++s) {
    int r, k;
    unit_source<BFAST, BN, CPR, Cfg::LINES>(s * NT + 64 * wave + lane, r, k);
    b_off[s] = offset(BFastT(), r, k, n_left, g.ldb);
  }
  // The resources of the slab from k0 (< K) on.
  auto rsrc_a = [&](int k0) {
    return AFAST ? rsrc_slab_a(At, a_cap, k0) : rsrc_at(At, a_rem, (int64_t)k0 * g.lda);
  };
  auto rsrc_b = [&](int k0) {
    return BFAST ? rsrc_slab_a(Bt, b_cap, k0) : rsrc_at(Bt, b_rem, (int64_t)k0 * g.ldb);
  };

  auto issue_one = [&](int l, __amdgpu_buffer_rsrc_t qa, __amdgpu_buffer_rsrc_t qb, int st) {
#pragma unroll
    for (int s = 0; s < Cfg::A_SLOTS; ++s)
      if (l == s) load4_to_lds(qa, As + st * Cfg::A_STAGE + 4 * (s * NT + 64 * wave), a_off[s]);
#pragma unroll
    for (int s = 0; s < Cfg::B_SLOTS; ++s)
      if (l == Cfg::A_SLOTS + s)
        load4_to_lds(qb, Bs + st * Cfg::B_STAGE + 4 * (s * NT + 64 * wave), b_off[s]);
  };
  auto issue = [&](__amdgpu_buffer_rsrc_t qa, __amdgpu_buffer_rsrc_t qb, int st) {
#pragma unroll
    for (int l = 0; l < Cfg::LOADS; ++l) issue_one(l, qa, qb, st);
  };

  f32x16 acc[TA][TB];
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  const int nslab = (K + BK - 1) / BK;
  const bool k_tail = (AFAST || BFAST) && K % BK != 0;

  // Zeroes this lane's own words at k >= K of slab t once they have landed
  // (operands with k fast; the unit is worked out again here).
  auto fix_one = [&](auto fast, auto extent, float* stage, int slots, int left, int t) {
    if constexpr (decltype(fast)::value) {
      int ln = lane;
      asm volatile("" : "+v"(ln));
#pragma unroll
      for (int s = 0; s < slots; ++s) {
        int r, k;
        unit_source<true, decltype(extent)::value, CPR, Cfg::LINES>(s * NT + 64 * wave + ln, r, k);
        k += t * BK;
        if (k + 4 > K && r < left) {
          f32x4* unit = reinterpret_cast<f32x4*>(stage + 4 * (s * NT + 64 * wave + ln));
          f32x4 v = *unit;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (k + e >= K) v[e] = 0.0f;
          *unit = v;
        }
      }
    }
  };
  auto fix_tail = [&](int t, int st) {
    fix_one(AFastT(), std::integral_constant<int, BM>(), As + st * Cfg::A_STAGE, Cfg::A_SLOTS,
            m_left, t);
    fix_one(BFastT(), std::integral_constant<int, BN>(), Bs + st * Cfg::B_STAGE, Cfg::B_SLOTS,
            n_left, t);
  };

  constexpr bool kSpread = KS == 1;
  constexpr int NCH = 2 * SUB_G;
  struct Frag {
    f32x4 a[TA], b[TB];   // 4 k steps
  };
  // One operand's fragments of chunk c: k steps 4 (c & 1) .. + 3 of the wave
  // group's sub-slab c >> 1, lanes 32-63 eight further on.
  auto read_one = [&](auto fast, auto extent, f32x4* out, int T, const float* stage, int w0,
                      int sub, int h) {
    constexpr int R = decltype(extent)::value;
    if constexpr (decltype(fast)::value) {
      // Either layout repeats every 32 rows.
      const int c = 4 * sub + 2 * lh + h;
      const int unit = Cfg::LINES ? (w0 + li) * CPR + (c ^ fast_swizzle<CPR>(li))
                                  : w0 * CPR + (li >> 4) * (16 * CPR) + (li & 15) + 16 * c;
#pragma unroll
      for (int i = 0; i < T; ++i)
        out[i] = *reinterpret_cast<const f32x4*>(stage + 4 * (unit + 32 * i * CPR));
    } else {
      // One lane offset (two for R = 32, whose xor moves to the neighbouring
      // row), so that the k steps are immediates of the reads.
      const int col = T == 2 ? w0 + 2 * li : w0 + li;
      const int q = R >= 64 ? (col >> 2) ^ (lh ? 8 : 0) : col >> 2;
      const float* const p = stage + 4 * (8 * lh * (R / 4) + q) + (col & 3);
      const int flip = R >= 64 ? 0 : lh * R;
#pragma unroll
      for (int pp = 0; pp < 4; ++pp) {
        const float* const at = p + (16 * sub + 4 * h + pp) * R + (pp & 1 ? -flip : flip);
        if (T == 2) {
          const f32x2 v = *reinterpret_cast<const f32x2*>(at);
          out[0][pp] = v[0];
          out[T - 1][pp] = v[1];
        } else {
          out[0][pp] = *at;
        }
      }
    }
  };
  auto read_chunk = [&](Frag& f, int st, int c) {
    const int sub = grp * SUB_G + (c >> 1), h = c & 1;
    read_one(AFastT(), std::integral_constant<int, BM>(), f.a, TA, As + st * Cfg::A_STAGE, wm0,
             sub, h);
    read_one(BFastT(), std::integral_constant<int, BN>(), f.b, TB, Bs + st * Cfg::B_STAGE, wn0,
             sub, h);
  };
  auto mfma_chunk = [&](const Frag& f, auto loads, __amdgpu_buffer_rsrc_t qa,
                        __amdgpu_buffer_rsrc_t qb, int st, auto pin_first) {
#pragma unroll
    for (int pp = 0; pp < 4; ++pp) {
      if constexpr (decltype(loads)::value) {
#pragma unroll
        for (int l = 0; l < Cfg::LOADS; ++l)
          if (pp == l * 4 / Cfg::LOADS) issue_one(l, qa, qb, st);
      }
#pragma unroll
      for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(f.a[i][pp], f.b[j][pp], acc[i][j], 0,
                                                           0, 0);
      if constexpr (decltype(pin_first)::value)
        if (pp == 0) __builtin_amdgcn_sched_barrier(0);
    }
  };
  Frag fr[2];
  const __amdgpu_buffer_rsrc_t qz = make_rsrc(g.A, 0u);
  auto chunks = [&](int st) {
#pragma unroll
    for (int c = 0; c + 1 < NCH; ++c) {
      read_chunk(fr[(c + 1) & 1], st, c + 1);
      __builtin_amdgcn_sched_barrier(0);
      mfma_chunk(fr[c & 1], std::false_type(), qz, qz, 0,
                 std::integral_constant<bool, KS == 4>());
    }
  };
  // Slab t (in stage t mod S) when a slab t + 1 follows; with LOADS slab t + S is
  // loaded into the stage that slab t leaves, and slabs t + 2 .. t + S - 1 stay
  // in flight across the wait.
  auto step = [&](int t, auto loads) {
    constexpr bool kLoads = decltype(loads)::value;
    const int st = t % S, nst = (t + 1) % S;
    __amdgpu_buffer_rsrc_t qa = qz, qb = qz;
    if constexpr (kLoads) {
      qa = rsrc_a((t + S) * BK);
      qb = rsrc_b((t + S) * BK);
    }
    chunks(st);
    if constexpr (KS == 2) __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(kWaitLoads<kLoads ? (S - 2) * Cfg::LOADS : 0>);
    if (k_tail && t + 2 == nslab) fix_tail(t + 1, nst);
    __builtin_amdgcn_s_waitcnt(kWaitLds);
    asm volatile("s_barrier" ::: "memory");
    if constexpr (kSpread) {
      read_chunk(fr[0], nst, 0);
      __builtin_amdgcn_sched_barrier(0);
      mfma_chunk(fr[1], loads, qa, qb, st, std::false_type());
    } else {
      if constexpr (kLoads) issue(qa, qb, st);
      read_chunk(fr[0], nst, 0);
      __builtin_amdgcn_sched_barrier(0);
      mfma_chunk(fr[1], std::false_type(), qz, qz, st, std::false_type());
    }
  };
  // A wave whose part of the tile lies outside C only loads: its share of the
  // matrix pipe goes to the others, so an edge tile costs what its waves with
  // work cost.
  const bool works = wm0 < m_left && wn0 < n_left;
  if (nslab > 0) {
    // Slabs 0 .. S-2 go out at once; slab 0 is waited for (with those behind it
    // when there are fewer), published, and slab S-1 goes out.
    issue(rsrc_a(0), rsrc_b(0), 0);
#pragma unroll
    for (int j = 1; j + 1 < S; ++j)
      if (j < nslab) issue(rsrc_a(j * BK), rsrc_b(j * BK), j);
    if (nslab >= S - 1)
      __builtin_amdgcn_s_waitcnt(kWaitLoads<(S - 2) * Cfg::LOADS>);
    else
      __builtin_amdgcn_s_waitcnt(kWaitLoads<0>);
    if (k_tail && nslab == 1) fix_tail(0, 0);
    __builtin_amdgcn_s_waitcnt(kWaitLds);
    asm volatile("s_barrier" ::: "memory");
    if (nslab > S - 1) issue(rsrc_a((S - 1) * BK), rsrc_b((S - 1) * BK), S - 1);
    if (works) {
      read_chunk(fr[0], 0, 0);
      int t = 0;
      for (; t + S < nslab; ++t) step(t, std::true_type());
      if constexpr (S == 2) {
        if (t + 1 < nslab) {
          step(t, std::false_type());
          ++t;
        }
      } else {
        for (; t + 1 < nslab; ++t) step(t, std::false_type());
      }
      chunks(t % S);
      mfma_chunk(fr[1], std::false_type(), qz, qz, 0, std::false_type());
    } else {
      // The same waits and barriers.
      for (int t = 0; t + 1 < nslab; ++t) {
        if (t + S < nslab)
          __builtin_amdgcn_s_waitcnt(kWaitLoads<(S - 2) * Cfg::LOADS>);
        else
          __builtin_amdgcn_s_waitcnt(kWaitLoads<0>);
        if (k_tail && t + 2 == nslab) fix_tail(t + 1, (t + 1) % S);
        __builtin_amdgcn_s_waitcnt(kWaitLds);
        asm volatile("s_barrier" ::: "memory");
        if (t + S < nslab) issue(rsrc_a((t + S) * BK), rsrc_b((t + S) * BK), t % S);
      }
    }
  }
  // Every wave has read its last fragments before LDS is used again.
  __syncthreads();

  if constexpr (KS > 1) {
    // Groups 1..KS-1 leave their partial tiles in LDS and group 0 adds them in
    // group order.
    constexpr int PER_WAVE = TA * TB * 16 * 64;
    if (grp > 0) {
      float* dst = lds + ((grp - 1) * Cfg::SPATIAL + sw) * PER_WAVE + lane;
#pragma unroll
      for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) dst[((i * TB + j) * 16 + r) * 64] = acc[i][j][r];
    }
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int q = 1; q < KS; ++q) {
        const float* src = lds + ((q - 1) * Cfg::SPATIAL + sw) * PER_WAVE + lane;
#pragma unroll
        for (int i = 0; i < TA; ++i)
#pragma unroll
          for (int j = 0; j < TB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] += src[((i * TB + j) * 16 + r) * 64];
      }
    }
    __syncthreads();   // the sums are read before the rows below overwrite them
    if (grp > 0) return;
  }

  // The epilogue, 32 rows of the wave tile at a time.
  int ln = lane;
  asm volatile("" : "+v"(ln));
  const int col = 4 * (ln % LPR);              // from the wave's first column
  const int cols = n_left - wn0 - col;         // left of this lane's column
  float* const rows = lds + sw * 32 * WN;
  float* out;
  int ld_out;
  if (partial) {
    const int64_t plane = (int64_t)g.M * g.N;
    out = g.W + (g.mode == kSumGroups ? (int64_t)split * g.groups + group : split) * plane +
          (int64_t)row0 * g.N;
    ld_out = g.N;
  } else {
    out = g.C + (g.mode == kSumGroups ? group * g.stride_c : 0) + (int64_t)row0 * g.ldc;
    ld_out = g.ldc;
  }
  out += n0;
  float* pre = partial || !g.preact ? nullptr : g.preact + (int64_t)row0 * g.ldp + n0;
  if (!kEarly) load_bias(ln);
  const int act = partial ? SGEMM_ACT_NONE : g.act;
#pragma unroll
  for (int i = 0; i < TA; ++i) {
    const int li_c = ln & 31, lh_c = ln >> 5;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float* p = rows + (8 * (r >> 2) + 4 * lh_c + (r & 3)) * WN;
      if constexpr (kPairB) {
        const f32x2 v = {acc[i][0][r], acc[i][TB - 1][r]};
        *reinterpret_cast<f32x2*>(p + 2 * li_c) = v;
      } else {
#pragma unroll
        for (int j = 0; j < TB; ++j) p[32 * j + li_c] = acc[i][j][r];
      }
    }
    if (!kEarly) load_residual(i, ln);
    // This wave's own part of LDS: its writes above, then its reads below.
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    f32x4* const mine = reinterpret_cast<f32x4*>(rows) + ln;
    // A bias alone is added with the residual.
    const bool through = act != SGEMM_ACT_NONE || pre;
    if (through) {
      with_activation(act, [&](auto which) {
        constexpr int kRounds = kEarly ? 2 : 1;
#pragma unroll kRounds
        for (int it = 0; it < IT; ++it) {
          f32x4 z = mine[it * 64];
          z += bias;
          if (pre) {
            const int row = row_of(i, it * RPI + ln / LPR);
            if (row < m_left && cols > 0)
              store_upto_once(pre + (uint32_t)row * (uint32_t)g.ldp + (uint32_t)(wn0 + col), cols,
                              z);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) z[e] = activate<decltype(which)::value>(z[e]);
          mine[it * 64] = z;
        }
      });
    }
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int row = row_of(i, it * RPI + ln / LPR);
      if (row < m_left && cols > 0) {
        f32x4 v = mine[it * 64];
        if (!through) v += bias;
        if (res) v += add[it];
        float* const p = out + (uint32_t)row * (uint32_t)ld_out + (uint32_t)(wn0 + col);
        if (partial) store_upto(p, cols, v);
        else store_upto_once(p, cols, v);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

}  // namespace sg
