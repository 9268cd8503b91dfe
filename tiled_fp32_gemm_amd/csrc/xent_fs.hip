// xent_fs.hip -- the cross entropy's products for B stored H x V.
#include "xent_table.hpp"

namespace sg {

const XentVariant* xent_variants_fs() { return xent_variants<false>(); }

}  // namespace sg
