// xent_ff.hip -- the cross entropy's products for B stored V x H.
#include "xent_table.hpp"

namespace sg {

const XentVariant* xent_variants_ff() { return xent_variants<true>(); }

}  // namespace sg
