// oz2_linear_gemm.hip -- which kernel a linear-layer product runs on, and the packing of
// operands whose rows are not aligned.  The kernels are in oz2_linear_tile.hpp.
#include <algorithm>

#include "oz2_common.hpp"
#include "oz2_linear.hpp"

namespace oz2 {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// The plan with the least estimated time, in microseconds.  Measured on bf16 products of 8 to
// 8192 rows, 1024 to 8192 columns and depths 512 to 8192 (the estimates are within 15% there):
//   a stage (128 bytes of depth) takes 1.5 on a 256 x 256 tile, one to a CU; 0.7 on a
//   128 x 128 tile alone on a CU and 0.5 each on two or more; 0.4 and 0.3 on a 64 x 128 tile;
//   a launch with its first loads and its epilogue 5, a join 3, and the partial sums' bytes
//   5 per 25 MB written and read.
// So few tiles on a long depth are split until the CUs are full, and no further.
Plan plan_product(bool i8, long rows, long cols, long depth, bool left_along_index, bool right_along_index) {
  constexpr long kCus = 256;
  Plan best{kTile128, 1};
  if (rows <= 0 || cols <= 0) return best;  // nothing to compute
  if (!left_along_index && !right_along_index && rows <= 16)
    return Plan{rows <= 8 ? kFew8 : kFew16, 1};
  const long stages = (depth * (i8 ? 1 : 2) + 127) / 128;
  auto tiles = [&](long m, long n) { return (rows + m - 1) / m * ((cols + n - 1) / n); };
  auto per_cu = [&](long n) { return (n + kCus - 1) / kCus; };
  double least = per_cu(tiles(256, 256)) * stages * 1.5 + 5.0;
  best.tile = kTile256;
  const bool low = rows <= 64 && !left_along_index;
  const long n = low ? tiles(64, 128) : tiles(128, 128);
  const double alone = low ? 0.4 : 0.7, shared = low ? 0.3 : 0.5;
  for (const int splits : {1, 2, 3, 4, 6, 8, 11, 16, 22, 32}) {
    if (splits > 1 && 2 * splits > stages) break;
    const long per = (stages + splits - 1) / splits;
    const long used = per > 0 ? (stages + per - 1) / per : 1;  // parts that are not empty
    const long load = per_cu(n * used);
    double t = per * (load == 1 ? alone : shared * load) + 5.0;
    if (used > 1) t += 3.0 + 8e-6 / 5.0 * used * rows * cols;
    if (t < least) {
      least = t;
      best = Plan{low ? kTile64 : kTile128, static_cast<int>(used)};
    }
  }
  return best;
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
