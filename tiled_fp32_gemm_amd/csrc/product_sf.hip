// product_sf.hip -- product_kernel's variants for A stored K x M, B stored N x K.
#include "product_table.hpp"

namespace sg {

const ProductVariant* product_variants_sf() { return product_variants<false, true>(); }

}  // namespace sg
