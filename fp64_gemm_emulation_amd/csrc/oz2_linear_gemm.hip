// oz2_linear_gemm.hip -- which kernel a linear-layer product runs on, and the packing of
// operands whose rows are not aligned.  The kernels are in oz2_linear_tile.hpp.
#include <algorithm>

#include "oz2_common.hpp"
#include "oz2_linear.hpp"

namespace oz2 {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// The plan with the least estimated time, in microseconds.  Measured on bf16 products of 17 to
// 8192 rows, 1024 to 8192 columns and depths 512 to 8192 (the estimates are within 15% there):
//   a stage (128 bytes of depth) takes 1.55 on a 256 x 256 tile, one to a CU; 0.45 on a
//   128 x 128 tile alone on a CU and 0.5 each on two or more; 0.27 on a 64 x 128 tile;
//   a launch with its first loads and its epilogue 5.5, a join 3, and the partial sums' bytes
//   5 per 25 MB written and read.
// So few tiles on a long depth are split until the CUs are full, and no further: 1024 x 2048
// outputs at depth 8192 take 60 in one part, 43.5 in two and 52.5 in four.
Plan plan_product(bool i8, long rows, long cols, long depth, bool left_along_index, bool right_along_index) {
  constexpr long kCus = 256;
  Plan best{kTile128, 1};
  if (rows <= 0 || cols <= 0) return best;  // nothing to compute
  if (!left_along_index && !right_along_index && rows <= 16)
    return Plan{rows <= 8 ? kFew8 : kFew16, 1};
  const long stages = (depth * (i8 ? 1 : 2) + 127) / 128;
  auto tiles = [&](long m, long n) { return (rows + m - 1) / m * ((cols + n - 1) / n); };
  auto per_cu = [&](long n) { return (n + kCus - 1) / kCus; };
  const long n128 = tiles(128, 128), n64 = tiles(64, 128);
  double least = per_cu(tiles(256, 256)) * stages * 1.55 + 5.5;
  best.tile = kTile256;
  const bool low = rows <= 64 && !left_along_index;
  for (const int splits : {1, 2, 3, 4, 6, 8, 11, 16, 22, 32}) {
    if (splits > 1 && 2 * splits > stages) break;
    const long per = (stages + splits - 1) / splits;
    const long used = per > 0 ? (stages + per - 1) / per : 1;  // parts that are not empty
    const double join = used > 1 ? 3.0 + 8e-6 / 5.0 * used * rows * cols : 0.0;
    auto consider = [&](int tile, double stage_time, long load) {
      const double t = per * stage_time * load + 5.5 + join;
      if (t >= least) return;
      least = t;
      best = Plan{tile, static_cast<int>(used)};
    };
    if (low) {
      consider(kTile64, 0.27, per_cu(n64 * used));
    } else {
      const long load = per_cu(n128 * used);
      consider(load == 1 ? kTile128Deep : kTile128, load == 1 ? 0.45 : 0.5, load);
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
