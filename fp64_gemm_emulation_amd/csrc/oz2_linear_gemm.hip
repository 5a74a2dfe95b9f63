// oz2_linear_gemm.hip -- which kernel a linear-layer product runs on, and the packing of
// operands whose rows are not aligned.  The kernels are in oz2_linear_tile.hpp.
#include <algorithm>

#include "oz2_common.hpp"
#include "oz2_linear.hpp"

namespace oz2 {

typedef int i32x4 __attribute__((ext_vector_type(4)));

Plan plan_product(bool i8, long rows, long cols, long depth, bool left_along_index, bool right_along_index) {
  Plan plan{kTile128, 1};
  if (rows <= 0 || cols <= 0) return plan;  // nothing to compute
  if (!left_along_index && !right_along_index && rows <= 32) {
    plan.tile = kFew;
    return plan;
  }
  const long t256 = (rows + 255) / 256 * ((cols + 255) / 256);
  if (t256 >= 192) {
    plan.tile = kTile256;
    return plan;
  }
  if (rows <= 64 && !left_along_index) plan.tile = kTile64;
  const long tiles = plan.tile == kTile64 ? (cols + 127) / 128 : (rows + 127) / 128 * ((cols + 127) / 128);
  const long stages = (depth * (i8 ? 1 : 2) + 127) / 128;
  // parts of at least four stages
  long splits = std::min(512 / tiles, stages / 4);
  if (splits > 1) {
    const long per = (stages + splits - 1) / splits;
    splits = (stages + per - 1) / per;  // none of them empty
  }
  plan.splits = static_cast<int>(std::max(1L, splits));
  return plan;
}

hipError_t launch_product(const Product& pr, hipStream_t st) {
  if (pr.i8) return launch_product_i8(pr, st);
  return pr.type == kTypeBf16 ? launch_product_bf16(pr, st) : launch_product_f16(pr, st);
}

// ---- packing ------------------------------------------------------------------------------
// Rows copied to a row stride of ld_out elements (a multiple of 8), zeros behind each row's end:
// for operands whose rows do not all start on 16-byte boundaries, which the tile kernel's
// copies need.  16 bytes per thread.
template <typename U>
__global__ __launch_bounds__(256) void pack_rows_kernel(long rows, int cols, const U* src, long ld, U* dst, long ld_out) {
  constexpr int N = 16 / sizeof(U);
  const int c = N * (blockIdx.y * 256 + threadIdx.x);
  if (c >= ld_out) return;
  for (long row = blockIdx.x; row < rows; row += gridDim.x) {
    U v[N];
    const U* const p = src + row * ld + c;
    if (c + N <= cols) {
      __builtin_memcpy(v, p, 16);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = c + i < cols ? p[i] : U(0);
    }
    *reinterpret_cast<i32x4*>(dst + row * ld_out + c) = __builtin_bit_cast(i32x4, v);
  }
}

hipError_t launch_pack_rows(int elem, long rows, int cols, const void* src, long ld, void* dst, long ld_out, hipStream_t st) {
  if (rows == 0 || cols == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(rows < (1 << 20) ? rows : (1 << 20)),
                  static_cast<unsigned>((ld_out / (16 / elem) + 255) / 256));
  if (elem == 1)
    hipLaunchKernelGGL(pack_rows_kernel<uint8_t>, grid, dim3(256), 0, st, rows, cols, static_cast<const uint8_t*>(src), ld,
                       static_cast<uint8_t*>(dst), ld_out);
  else
    hipLaunchKernelGGL(pack_rows_kernel<uint16_t>, grid, dim3(256), 0, st, rows, cols, static_cast<const uint16_t*>(src), ld,
                       static_cast<uint16_t*>(dst), ld_out);
  return hipGetLastError();
}

}  // namespace oz2
