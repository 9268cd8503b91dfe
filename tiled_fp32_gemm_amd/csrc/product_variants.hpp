// product_variants.hpp -- the tile variants of product_kernel, one table for
// each pair of operand layouts (product_*.hip compile one each).
#pragma once

#include "host.hpp"
#include "product_args.hpp"

namespace sg {

typedef void (*ProductFn)(ProductArgs);

struct ProductVariant {
  const char* name;
  host::TileCost cost;
  int lds_bytes;
  ProductFn fn;
};

constexpr int kProductVariants = 8;

// [A stored M x K][B stored N x K]
const ProductVariant* product_variants_ss();   // A is K x M, B is K x N
const ProductVariant* product_variants_sf();   // A is K x M, B is N x K
const ProductVariant* product_variants_fs();   // A is M x K, B is K x N
const ProductVariant* product_variants_ff();   // A is M x K, B is N x K

// kernel_rows.hpp: chunks of `rows` (1, 2, 4 or 8) rows; `cols` a workgroup are
// 16 or 4 with B stored N x K (KW 1 and 4), and 64, 32 or 16 with K x N.
constexpr int kRowsMost = 8;
ProductFn rows_kernel(bool b_fast, int rows, int cols, int threads, bool deep);

}  // namespace sg
