// product_ff.hip -- product_kernel's variants for A stored M x K, B stored N x K.
#include "product_table.hpp"

namespace sg {

const ProductVariant* product_variants_ff() { return product_variants<true, true>(); }

}  // namespace sg
