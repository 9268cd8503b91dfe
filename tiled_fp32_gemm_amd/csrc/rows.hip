// rows.hip -- the variants of kernel_rows.hpp.
#include "kernel_rows.hpp"
#include "product_variants.hpp"

namespace sg {

namespace {

template <int R>
ProductFn rows_variant(bool b_fast, int cols, int threads, bool deep) {
  constexpr bool kDeep = R >= 4;
  if (b_fast && deep && kDeep)
    return cols == 16 ? rows_fast_kernel<R, 4, 1, kDeep> : rows_fast_kernel<R, 4, 4, kDeep>;
  if (b_fast)
    return cols == 16 ? rows_fast_kernel<R, 4, 1, false> : rows_fast_kernel<R, 4, 4, false>;
  return cols == 16       ? rows_slow_kernel<R, 4, 512>
         : cols == 32     ? rows_slow_kernel<R, 8, 512>
         : threads == 512 ? rows_slow_kernel<R, 16, 512>
                          : rows_slow_kernel<R, 16, 256>;
}

}  // namespace

ProductFn rows_kernel(bool b_fast, int rows, int cols, int threads, bool deep) {
  return rows == 1   ? rows_variant<1>(b_fast, cols, threads, deep)
         : rows == 2 ? rows_variant<2>(b_fast, cols, threads, deep)
         : rows == 4 ? rows_variant<4>(b_fast, cols, threads, deep)
                     : rows_variant<8>(b_fast, cols, threads, deep);
}

}  // namespace sg
