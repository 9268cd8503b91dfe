// product_ss.hip -- product_kernel's variants for A stored K x M, B stored K x N.
#include "product_table.hpp"

namespace sg {

const ProductVariant* product_variants_ss() { return product_variants<false, false>(); }

}  // namespace sg
