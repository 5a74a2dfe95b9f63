// oz2_linear_f16.hip -- the linear-layer products on f16 operands.
#include "oz2_linear_tile.hpp"

namespace oz2 {

hipError_t launch_product_f16(const Product& pr, hipStream_t st) {
  return launch_type<MmaF16, f16>(pr, st);
}

hipError_t launch_pair_f16(const Product& dx, const Product& dw, const ColumnSums& sums, hipStream_t st) {
  return launch_pair<MmaF16, f16>(dx, dw, sums, st);
}

}  // namespace oz2
