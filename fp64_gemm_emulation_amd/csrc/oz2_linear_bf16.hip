// oz2_linear_bf16.hip -- the linear-layer products on bf16 operands.
#include "oz2_linear_tile.hpp"

namespace oz2 {

hipError_t launch_product_bf16(const Product& pr, hipStream_t st) {
  return launch_type<MmaBf16, bf16>(pr, st);
}

hipError_t launch_pair_bf16(const Product& dx, const Product& dw, const ColumnSums& sums, hipStream_t st) {
  return launch_pair<MmaBf16, bf16>(dx, dw, sums, st);
}

}  // namespace oz2
