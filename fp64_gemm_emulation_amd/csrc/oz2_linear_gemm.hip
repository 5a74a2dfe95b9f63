// oz2_linear_gemm.hip -- out = epilogue(left right^T), the products of the linear layer and of
// its gradient: bf16 and f16 operands with f32 accumulators, int8 operands with int32 ones
// (exact: 127^2 times the depth stays below 2^31 up to the 2^17 the entry points accept).
#include "oz2_common.hpp"
#include "oz2_linear.hpp"

namespace oz2 {

typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// One 16 x 16 block over 64 bytes of depth per operand row: 32 16-bit or 64 int8 elements,
// lane l holding 16 bytes of row l % 16.  D register v of lane l is row 4 (l / 16) + v of the
// first operand and row l % 16 of the second.
struct MmaBf16 {
  typedef bf16 elem;
  typedef f32x4 acc;
  static __device__ __forceinline__ acc mma(i32x4 a, i32x4 b, acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
struct MmaF16 {
  typedef f16 elem;
  typedef f32x4 acc;
  static __device__ __forceinline__ acc mma(i32x4 a, i32x4 b, acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
struct MmaI8 {
  typedef int8_t elem;
  typedef i32x4 acc;
  static __device__ __forceinline__ acc mma(i32x4 a, i32x4 b, acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
};

// The simplest form: a 64 x 64 output tile per workgroup, 64 bytes of depth at a time, single
// elements through registers into shared memory, any strides.
template <typename M, typename T>
__global__ __launch_bounds__(256) void product_simple_kernel(int rows, int cols, int depth,
                                                             const typename M::elem* __restrict__ left, long left_row,
                                                             long left_step, const typename M::elem* __restrict__ right,
                                                             long right_row, long right_step, Epilogue e) {
  typedef typename M::elem E;
  constexpr int BK = 64 / sizeof(E);
  __shared__ __attribute__((aligned(16))) E sl[64][BK];
  __shared__ __attribute__((aligned(16))) E sr[64][BK];
  __shared__ float out[64][65];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const unsigned tiles_n = (static_cast<unsigned>(cols) + 63) / 64;
  const long m0 = static_cast<long>(blockIdx.x / tiles_n) * 64;
  const int n0 = static_cast<int>(blockIdx.x % tiles_n) * 64;
  typename M::acc acc[4] = {};
  for (int k0 = 0; k0 < depth; k0 += BK) {
    for (int i = tid; i < 64 * BK; i += 256) {
      const int row = i / BK, k = i % BK;
      const bool in_k = k0 + k < depth;
      sl[row][k] = in_k && m0 + row < rows ? left[(m0 + row) * left_row + (k0 + k) * left_step] : E(0);
      sr[row][k] = in_k && n0 + row < cols ? right[(n0 + row) * right_row + (k0 + k) * right_step] : E(0);
    }
    __syncthreads();
    const int k16 = (lane >> 4) * (16 / static_cast<int>(sizeof(E)));
    const i32x4 b = *reinterpret_cast<const i32x4*>(&sl[16 * wave + (lane & 15)][k16]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc[j] = M::mma(*reinterpret_cast<const i32x4*>(&sr[16 * j + (lane & 15)][k16]), b, acc[j]);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) out[16 * wave + (lane & 15)][16 * j + 4 * (lane >> 4) + v] = static_cast<float>(acc[j][v]);
  __syncthreads();
  for (int g = tid; g < 64 * 8; g += 256) {
    const int row = g >> 3, n = n0 + 8 * (g & 7);
    if (m0 + row >= rows || n >= cols) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = out[row][8 * (g & 7) + i];
    finish8<T>(v, e, m0 + row, n, cols);
  }
}

template <typename M, typename T>
static hipError_t launch_simple(const Product& pr, hipStream_t st) {
  typedef typename M::elem E;
  const dim3 grid(static_cast<unsigned>((pr.cols + 63) / 64) * static_cast<unsigned>((pr.rows + 63) / 64));
  hipLaunchKernelGGL((product_simple_kernel<M, T>), grid, dim3(256), 0, st, pr.rows, pr.cols, pr.depth,
                     static_cast<const E*>(pr.left), pr.left_row, pr.left_step, static_cast<const E*>(pr.right),
                     pr.right_row, pr.right_step, pr.epi);
  return hipGetLastError();
}

hipError_t launch_product(const Product& pr, hipStream_t st) {
  if (pr.i8) return pr.type == kTypeBf16 ? launch_simple<MmaI8, bf16>(pr, st) : launch_simple<MmaI8, f16>(pr, st);
  return pr.type == kTypeBf16 ? launch_simple<MmaBf16, bf16>(pr, st) : launch_simple<MmaF16, f16>(pr, st);
}

}  // namespace oz2
