// product_table.hpp -- instantiates product_kernel's tiles for one pair of
// operand layouts.  The rates and occupancies are those of the same tiles in
// sgemm.hip, whose main loop is the same.
#pragma once

#include "kernel_product.hpp"
#include "product_variants.hpp"

namespace sg {

template <int BM, int BN, int WM, int WN, int BK, int KS, bool AF, bool BF>
ProductVariant product_variant(const char* name, double eff, int occ) {
  using Cfg = ProductCfg<BM, BN, WM, WN, BK, KS>;
  return {name, {BM, BN, BK, Cfg::NT, eff, occ}, Cfg::LDS_FLOATS * 4,
          product_kernel<BM, BN, WM, WN, BK, KS, AF, BF>};
}

template <bool AF, bool BF>
const ProductVariant* product_variants() {
  static const ProductVariant table[kProductVariants] = {
      product_variant<256, 256, 64, 64, 32, 1, AF, BF>("256x256x32", 0.929, 1),
      product_variant<128, 128, 32, 64, 32, 1, AF, BF>("128x128x32", 0.895, 2),
      product_variant<64, 128, 32, 64, 32, 1, AF, BF>("64x128x32", 0.901, 3),
      product_variant<64, 128, 32, 64, 32, 2, AF, BF>("64x128x32_ks2", 0.805, 3),
      product_variant<64, 64, 32, 32, 32, 1, AF, BF>("64x64x32", 0.837, 5),
      product_variant<64, 64, 32, 32, 32, 2, AF, BF>("64x64x32_ks2", 0.830, 4),
      product_variant<32, 64, 32, 32, 32, 2, AF, BF>("32x64x32_ks2", 0.799, 6),
      product_variant<32, 64, 32, 32, 64, 4, AF, BF>("32x64x64_ks4", 0.807, 3)};
  return table;
}

}  // namespace sg
