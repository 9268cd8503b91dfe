// product_table.hpp -- instantiates product_kernel's tiles for one pair of
// operand layouts.  The rates, slab times and occupancies are fitted to 43
// shapes (17 to 65536 rows, 100^3 to 4096^3) in all four layouts, each with
// every tile and up to sixteen splits of K: the choice is 1% behind the fastest
// on average, 6% at worst; the four layouts need no figures of their
// own.  "s4" keeps three slabs in flight, for grids that leave CUs with a
// workgroup or two, where a slab costs its loads' latency.
#pragma once

#include "kernel_product.hpp"
#include "product_variants.hpp"

namespace sg {

template <int BM, int BN, int WM, int WN, int BK, int KS, int ST, bool AF, bool BF>
ProductVariant product_variant(const char* name, double eff, int occ, double slab_floor,
                               double saturate = 1.0, double round_more = 0.0) {
  using Cfg = ProductCfg<BM, BN, WM, WN, BK, KS, ST>;
  return {name, {BM, BN, BK, Cfg::NT, eff, occ, slab_floor, saturate, round_more}, Cfg::LDS_FLOATS * 4,
          product_kernel<BM, BN, WM, WN, BK, KS, ST, AF, BF>};
}

template <bool AF, bool BF>
const ProductVariant* product_variants() {
  static const ProductVariant table[kProductVariants] = {
      product_variant<256, 256, 64, 64, 32, 1, 2, AF, BF>("256x256x32", 0.960, 1, 0.64e-6, 1.28),
      product_variant<128, 128, 32, 64, 32, 1, 2, AF, BF>("128x128x32", 0.945, 2, 0.74e-6, 1.28),
      product_variant<64, 128, 32, 64, 32, 1, 2, AF, BF>("64x128x32", 0.940, 3, 0.50e-6, 1.28),
      product_variant<64, 128, 32, 64, 32, 2, 2, AF, BF>("64x128x32_ks2", 0.885, 3, 0.44e-6),
      product_variant<64, 64, 32, 32, 32, 1, 2, AF, BF>("64x64x32", 0.915, 5, 0.50e-6),
      product_variant<32, 64, 32, 32, 32, 2, 2, AF, BF>("32x64x32_ks2", 0.840, 6, 0.34e-6, 1.28),
      product_variant<32, 64, 32, 32, 64, 4, 2, AF, BF>("32x64x64_ks4", 0.855, 3, 0.56e-6, 1.0,
                                                        0.25e-6),
      product_variant<32, 64, 32, 32, 32, 2, 4, AF, BF>("32x64x32_ks2_s4", 0.840, 3, 0.32e-6)};
  return table;
}

}  // namespace sg
