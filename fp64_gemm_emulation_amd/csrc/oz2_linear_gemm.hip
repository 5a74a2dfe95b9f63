// oz2_linear_gemm.hip -- which kernel a linear-layer product runs on, and the packing of
// operands whose rows are not aligned.  The kernels are in oz2_linear_tile.hpp.
#include <algorithm>
#include <cmath>

#include "oz2_common.hpp"
#include "oz2_linear.hpp"

namespace oz2 {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr long kCus = 256;
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 11, 16, 22, 32};

static long ceil_div(long a, long b) { return (a + b - 1) / b; }

// A product on tiles of one size, its depth in parts of `per` stages.
struct Parts {
  long stages, per, used;  // used: parts that are not empty
  Parts(long stages, int splits) : stages(stages), per(ceil_div(stages, splits)), used(per > 0 ? ceil_div(stages, per) : 1) {}
  // join launch and the partial sums' bytes
  double join(long rows, long cols) const { return used > 1 ? 3.0 + 8e-6 / 5.0 * used * rows * cols : 0.0; }
};

// Estimated times in microseconds, from bf16 products with columns in whole vectors: a stage
// (128 bytes of depth) takes 1.55 on a 256 x 256 tile, one to a CU; 0.45 on a 128 x 128 tile
// alone on a CU (0.52 with an operand along the index) and 0.5 each on two or more; 0.27 on a
// 64 x 128 tile; a launch with its first loads and its epilogue 5.5, a join 3, and the partial
// sums' bytes 5 per 25 MB written and read.  Of 72 products of 32 to 8192 rows, 1000 to 8192
// columns and depths 512 to 8192 timed against them, gradients take 0.91 to 1.12 of the estimate;
// forward in 16 bits 0.9 to 1.1, but 0.73 to 0.83 with 32 and 100 rows and 1.2 at depth 512 on
// 256 x 256 tiles; int8 0.76 to 1.33 (1.25 and more where one round of 128 x 128 tiles takes most
// CUs).  Odd columns, whose stores the estimate leaves out, add up to 16%, and a third on
// 256 x 256 tiles.
constexpr double kLaunch = 5.5;
static double alone128(bool along_index) { return along_index ? 0.52 : 0.45; }

// The plan with the least estimated time.  Few tiles on a long depth are split until the CUs
// are full, and no further: 1024 x 2048 outputs at depth 8192 take 60 us in one part, 43.5 in
// two and 52.5 in four.
static Plan plan_tiles(bool i8, long rows, long cols, long depth, bool left_along_index, bool right_along_index, double* time) {
  Plan best{kTile256, 1};
  const long stages = ceil_div(depth * (i8 ? 1 : 2), 128);
  const long n128 = ceil_div(rows, 128) * ceil_div(cols, 128), n64 = ceil_div(rows, 64) * ceil_div(cols, 128);
  double least = ceil_div(ceil_div(rows, 256) * ceil_div(cols, 256), kCus) * stages * 1.55 + kLaunch;
  const bool low = rows <= 64 && !left_along_index;
  for (const int splits : kSplits) {
    if (splits > 1 && 2 * splits > stages) break;
    const Parts parts(stages, splits);
    auto consider = [&](int tile, double stage_time, long load) {
      const double t = parts.per * stage_time * load + kLaunch + parts.join(rows, cols);
      if (t >= least) return;
      least = t;
      best = Plan{tile, static_cast<int>(parts.used)};
    };
    if (low) {
      consider(kTile64, 0.27, ceil_div(n64 * parts.used, kCus));
    } else {
      const long load = ceil_div(n128 * parts.used, kCus);
      consider(load == 1 ? kTile128Deep : kTile128, load == 1 ? alone128(left_along_index || right_along_index) : 0.5, load);
    }
  }
  *time = least;
  return best;
}

Plan plan_product(bool i8, long rows, long cols, long depth, bool left_along_index, bool right_along_index) {
  if (rows <= 0 || cols <= 0) return Plan{kTile128, 1};  // nothing to compute
  double time;
  const Plan tiles = plan_tiles(i8, rows, cols, depth, left_along_index, right_along_index, &time);
  if (left_along_index || right_along_index || rows > 16) return tiles;
  // Few rows.  Eight rows of weights a workgroup give twice the workgroups, sixteen fetch the
  // left operand half as often: one row, 2048 x 8192 weights 8.6 us against 11.5; eight rows,
  // 4096 x 4096 weights 10.6 against 8.8.
  const double bytes = static_cast<double>(cols) * depth * (i8 ? 1 : 2);
  if (rows <= 8) {
    // workgroups that quantise: no more than are resident at once (18.0 us with 1024 of them,
    // 14.5 with 512)
    if (i8 && quantize_in_product(Plan{kFew8, 1}, rows, depth)) return Plan{cols > 16 * kCus ? kFew16 : kFew8, 1};
    const bool eight = rows <= 4 || cols < 16 * kCus || bytes / cols <= 4096;
    return Plan{eight ? kFew8 : kFew16, 1};
  }
  // 9 to 16 rows: the weights at 7.5 MB/us, slowed by the left operand's reads beside them and
  // by too few workgroups, against a tile's time or its weights at 5.2 MB/us
  const double few = 4.5 + bytes / 7.5e6 * (1.0 + rows / 24.0) * std::sqrt(std::max(1.0, 16.0 * kCus / cols));
  return few < std::max(time, 4.0 + bytes / 5.2e6) ? Plan{kFew16, 1} : tiles;
}

// Together the two products take the longer one's parts, or their whole work over all CUs if
// that is more; apart, the sum of their times.
bool plan_pair(long p, long q, long r, Plan& dx, Plan& dw) {
  dx = plan_product(false, p, q, r, false, true);
  dw = plan_product(false, r, q, p, true, true);
  if (p <= 0 || q <= 0 || r <= 0) return false;
  double tx, tw;
  plan_tiles(false, p, q, r, false, true, &tx);
  plan_tiles(false, r, q, p, true, true, &tw);
  double least = tx + tw + 2.0;  // a launch saved, and the column sums'
  const long nx = ceil_div(p, 128) * ceil_div(q, 128), nw = ceil_div(r, 128) * ceil_div(q, 128);
  if (nx + nw > 2 * kCus) return false;
  bool paired = false;
  for (const int sx : kSplits) {
    const Parts x(ceil_div(2 * r, 128), sx);
    if (sx > 1 && 2 * sx > x.stages) break;
    for (const int sw : kSplits) {
      const Parts w(ceil_div(2 * p, 128), sw);
      if (sw > 1 && 2 * sw > w.stages) break;
      const double load = static_cast<double>(nx * x.used * x.per + nw * w.used * w.per) / kCus;
      const double longest = static_cast<double>(std::max(x.per, w.per) * ceil_div(nx * x.used + nw * w.used, kCus));
      const double t = alone128(true) * std::max(load, longest) + kLaunch + x.join(p, q) + w.join(r, q);
      if (t >= least) continue;
      least = t;
      paired = true;
      dx = Plan{kTile128Deep, static_cast<int>(x.used)};
      dw = Plan{kTile128Deep, static_cast<int>(w.used)};
    }
  }
  return paired;
}

hipError_t launch_product_pair(int type, const Product& dx, const Product& dw, const ColumnSums& sums, hipStream_t st) {
  return type == kTypeBf16 ? launch_pair_bf16(dx, dw, sums, st) : launch_pair_f16(dx, dw, sums, st);
}

hipError_t launch_product(const Product& pr, hipStream_t st) {
  if (pr.i8) return launch_product_i8(pr, st);
  return pr.type == kTypeBf16 ? launch_product_bf16(pr, st) : launch_product_f16(pr, st);
}

hipError_t launch_product_adapters(const Product& pr, const Adapters& ad, hipStream_t st) {
  return pr.type == kTypeBf16 ? launch_adapters_bf16(pr, ad, st) : launch_adapters_f16(pr, ad, st);
}

// ---- packing ------------------------------------------------------------------------------
// Rows copied to a row stride of ld_out elements (a multiple of 16 bytes), zeros behind each
// row's end: for operands whose rows do not all start on 16-byte boundaries, which the tile
// kernel's copies need.  16 bytes per thread; one or two operands, the second's workgroups
// behind the first's.  777 x 1999 and 4099 x 1999 elements in 8.5 us, 4.6 TB/s.
template <typename U>
__device__ __forceinline__ void pack_rows(unsigned wg, unsigned workgroups, const PackJob& job) {
  constexpr int N = 16 / sizeof(U);
  const U* const src = static_cast<const U*>(job.src);
  U* const dst = static_cast<U*>(job.dst);
  const unsigned per_row = static_cast<unsigned>(job.ld_out / N);
  // (rows, cols below 2^23 and N >= 8: the chunk number fits 64 bits, a row's 32)
  for (unsigned long n = wg * 256ul + threadIdx.x; n < job.rows * per_row; n += workgroups * 256ul) {
    const long row = static_cast<long>(n / per_row);
    const int c = N * static_cast<int>(n % per_row);
    U v[N];
    const U* const p = src + row * job.ld + c;
    if (c + N <= job.cols) {
      __builtin_memcpy(v, p, 16);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = c + i < job.cols ? p[i] : U(0);
    }
    *reinterpret_cast<i32x4*>(dst + row * job.ld_out + c) = __builtin_bit_cast(i32x4, v);
  }
}

template <typename U>
__global__ __launch_bounds__(256) void pack_rows_kernel(unsigned first, PackJob a, PackJob b) {
  if (blockIdx.x < first)
    pack_rows<U>(blockIdx.x, first, a);
  else
    pack_rows<U>(blockIdx.x - first, gridDim.x - first, b);
}

hipError_t launch_pack_rows(int elem, const PackJob* a, const PackJob* b, hipStream_t st) {
  // four chunks a thread where there are many
  auto workgroups = [&](const PackJob* j) -> unsigned {
    if (j == nullptr || j->rows == 0 || j->cols == 0) return 0;
    const long chunks = j->rows * (j->ld_out * elem / 16);
    return static_cast<unsigned>(std::min(ceil_div(chunks, 256), std::max(4096L, ceil_div(chunks, 1024))));
  };
  const unsigned na = workgroups(a), nb = workgroups(b);
  if (na + nb == 0) return hipSuccess;
  const PackJob none{};
  const PackJob &ja = na > 0 ? *a : none, &jb = nb > 0 ? *b : none;
  if (elem == 1)
    hipLaunchKernelGGL(pack_rows_kernel<uint8_t>, dim3(na + nb), dim3(256), 0, st, na, ja, jb);
  else
    hipLaunchKernelGGL(pack_rows_kernel<uint16_t>, dim3(na + nb), dim3(256), 0, st, na, ja, jb);
  return hipGetLastError();
}

}  // namespace oz2
