// product_table.hpp -- instantiates product_kernel's tiles for one pair of
// operand layouts.  The rates and occupancies are those of the same tiles in
// sgemm.hip, whose main loop is the same.  Two more keep three and two slabs in
// flight ("s4", "s3"), for grids that leave CUs with a workgroup or two, where
// a slab costs its loads' latency: 512 x 512 x 2048 takes 22.6 us with "s4"
// and 32.7 with two stages (24.6 and 43.6 with B stored N x K); on full grids
// they are a little behind, for the workgroups that their LDS keeps out.
#pragma once

#include "kernel_product.hpp"
#include "product_variants.hpp"

namespace sg {

template <int BM, int BN, int WM, int WN, int BK, int KS, int ST, bool AF, bool BF>
ProductVariant product_variant(const char* name, double eff, int occ, double slab_floor,
                               double saturate = host::kSaturate) {
  using Cfg = ProductCfg<BM, BN, WM, WN, BK, KS, ST>;
  return {name, {BM, BN, BK, Cfg::NT, eff, occ, slab_floor, saturate}, Cfg::LDS_FLOATS * 4,
          product_kernel<BM, BN, WM, WN, BK, KS, ST, AF, BF>};
}

template <bool AF, bool BF>
const ProductVariant* product_variants() {
  // The time of a slab whose loads are waited for, B from beyond the L2.
  constexpr double kLong = BF ? 0.80e-6 : 0.66e-6, kShort = AF && !BF ? 0.45e-6 : 0.61e-6,
                   kDeep = BF ? 1.20e-6 : 0.75e-6;
  // Both operands k slow: fewer LDS reads of 128 bits, which suits this tile.
  constexpr double kWide = AF || BF ? 0.895 : 0.925;
  static const ProductVariant table[kProductVariants] = {
      product_variant<256, 256, 64, 64, 32, 1, 2, AF, BF>("256x256x32", 0.929, 1, kLong),
      product_variant<128, 128, 32, 64, 32, 1, 2, AF, BF>("128x128x32", kWide, 2, kLong),
      product_variant<64, 128, 32, 64, 32, 1, 2, AF, BF>("64x128x32", 0.901, 3, kLong),
      product_variant<64, 128, 32, 64, 32, 2, 2, AF, BF>("64x128x32_ks2", 0.805, 3, kLong),
      product_variant<64, 64, 32, 32, 32, 1, 2, AF, BF>("64x64x32", 0.837, 5, kLong),
      product_variant<64, 64, 32, 32, 32, 2, 2, AF, BF>("64x64x32_ks2", 0.830, 4, kShort),
      product_variant<32, 64, 32, 32, 32, 2, 2, AF, BF>("32x64x32_ks2", 0.799, 6, kShort),
      product_variant<32, 64, 32, 32, 64, 4, 2, AF, BF>("32x64x64_ks4", 0.807, 3, kDeep),
      product_variant<64, 64, 32, 32, 32, 1, 3, AF, BF>("64x64x32_s3", 0.780, 3, 0.37e-6, 1.0),
      product_variant<32, 64, 32, 32, 32, 2, 4, AF, BF>("32x64x32_ks2_s4", 0.775, 3, 0.28e-6,
                                                        1.0)};
  return table;
}

}  // namespace sg
