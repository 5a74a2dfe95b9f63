// oz2_adapters_bf16.hip -- the linear-layer products with adapters on bf16 operands.
#include "oz2_linear_tile.hpp"

namespace oz2 {

hipError_t launch_adapters_bf16(const Product& pr, const Adapters& ad, hipStream_t st) {
  return launch_adapters<MmaBf16, bf16>(pr, ad, st);
}

}  // namespace oz2
