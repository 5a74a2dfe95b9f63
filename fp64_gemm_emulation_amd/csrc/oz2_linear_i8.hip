// oz2_linear_i8.hip -- the linear-layer products on int8 operands.
#include "oz2_linear_tile.hpp"

namespace oz2 {

hipError_t launch_product_i8(const Product& pr, hipStream_t st) {
  return pr.type == kTypeBf16 ? launch_type<MmaI8, bf16>(pr, st) : launch_type<MmaI8, f16>(pr, st);
}

}  // namespace oz2
