// oz2_adapters_f16.hip -- the linear-layer products with adapters on f16 operands.
#include "oz2_linear_tile.hpp"

namespace oz2 {

hipError_t launch_adapters_f16(const Product& pr, const Adapters& ad, hipStream_t st) {
  return launch_adapters<MmaF16, f16>(pr, ad, st);
}

}  // namespace oz2
