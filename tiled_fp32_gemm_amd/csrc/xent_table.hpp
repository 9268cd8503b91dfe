// xent_table.hpp -- instantiates product_kernel's tiles with the cross entropy's
// epilogues for one layout of B.  The costs are product_table.hpp's, and choose the
// fastest or within 3% of it for 1 to 8192 rows (13 products, each with every tile).
// Longer slabs come first where the model sees no difference, as for a few rows over a
// B that comes from memory: 16 rows, H = 1024, V = 32768, B V x H 36.5 us by slabs of
// 32, 36.0 with four of them in flight, 32.1 by slabs of 64.
#pragma once

#include "kernel_product.hpp"
#include "xent_finish.hpp"

namespace sg {

template <int BM, int BN, int WM, int WN, int BK, int KS, int ST, bool BF>
XentVariant xent_variant(double eff, int occ, double slab_floor, double saturate,
                         double round_more = 0.0) {
  using Cfg = ProductCfg<BM, BN, WM, WN, BK, KS, ST>;
  return {{BM, BN, BK, Cfg::NT, eff, occ, slab_floor, saturate, round_more}, WN,
          product_kernel<BM, BN, WM, WN, BK, KS, ST, true, BF, XentStats>,
          product_kernel<BM, BN, WM, WN, BK, KS, ST, true, BF, XentGrad>};
}

template <bool BF>
const XentVariant* xent_variants() {
  static const XentVariant table[kXentVariants] = {
      xent_variant<256, 256, 64, 64, 32, 1, 2, BF>(0.960, 1, 0.64e-6, 1.28),
      xent_variant<128, 128, 32, 64, 32, 1, 2, BF>(0.945, 2, 0.74e-6, 1.28),
      xent_variant<64, 128, 32, 64, 32, 1, 2, BF>(0.940, 3, 0.50e-6, 1.28),
      xent_variant<64, 64, 32, 32, 32, 1, 2, BF>(0.915, 5, 0.50e-6, 1.0),
      xent_variant<32, 64, 32, 32, 64, 4, 2, BF>(0.855, 3, 0.56e-6, 1.0, 0.25e-6),
      xent_variant<32, 64, 32, 32, 32, 2, 4, BF>(0.840, 3, 0.32e-6, 1.0),
      xent_variant<32, 64, 32, 32, 32, 2, 2, BF>(0.840, 6, 0.34e-6, 1.28)};
  return table;
}

}  // namespace sg
