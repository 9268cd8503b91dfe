// product_fs.hip -- product_kernel's variants for A stored M x K, B stored K x N.
#include "product_table.hpp"

namespace sg {

const ProductVariant* product_variants_fs() { return product_variants<true, false>(); }

}  // namespace sg
