// oz2_adapters.hip -- S = scale X A^T, the first product of the adapters beside a linear layer.
#include <algorithm>

#include "oz2_linear_tile.hpp"

namespace oz2 {

// Sixteen tokens and one of their adapters per workgroup, blockIdx.y the first of them that it
// takes (in the order of their first tokens) and blockIdx.z the part of the depth.  The matrix
// instruction's rows are 16 of the adapter's, its columns the tokens, and the waves share the depth
// in steps of 32 elements; operands go straight from memory to registers, kDeep steps of each
// under way.  Every column is computed and an adapter's own tokens are stored.  RB: blocks of 16
// rows that share the tokens' fragments; ranks above 64 take several passes.
constexpr int kSumWaves = 8;

template <typename M, typename T, int RB>
__global__ __launch_bounds__(64 * kSumWaves) void adapter_sums_kernel(int rows, int depth, int per, const T* __restrict__ x,
                                                                      long ldx, Adapters ad) {
  typedef typename M::acc Acc;
  constexpr int kDeep = RB == 1 ? 4 : 2;
  __shared__ Acc sums[kSumWaves][RB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lk = 8 * (lane >> 4);
  const long m0 = 16l * blockIdx.x;
  // the adapter of the lane's token, and the tokens that are the first of theirs
  int own = m0 + li < rows ? ad.index[m0 + li] : -1;
  if (own < 0 || own >= ad.count) own = -1;
  bool first = own >= 0 && lane < 16;
#pragma unroll
  for (int j = 0; j < 15; ++j) {
    const int before = __shfl(own, j, 64);
    first = first && (j >= li || before != own);
  }
  unsigned firsts = static_cast<unsigned>(__ballot(first));
  const int k_begin = per * static_cast<int>(blockIdx.z), k_end = min(k_begin + per, depth);
  const T* const xrow = x + min(m0 + li, static_cast<long>(rows) - 1) * ldx;
  const int pitch = ad.pitch();
  for (int n = 0; firsts != 0; ++n) {
    const int token = __builtin_ctz(firsts);
    firsts &= firsts - 1;
    if (n % gridDim.y != blockIdx.y) continue;
    const int adapter = __shfl(own, token, 64);
    for (int r0 = 0; r0 < ad.rank; r0 += 16 * RB) {
      const T* arow[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b)
        arow[b] = static_cast<const T*>(ad.a) + adapter * ad.stride_a + min(r0 + 16 * b + li, ad.rank - 1) * ad.lda;
      Acc acc[RB] = {};
      int k = k_begin + 32 * wave;
      for (; k + 32 * kSumWaves * (kDeep - 1) + 32 <= k_end; k += 32 * kSumWaves * kDeep) {
        i32x4 xv[kDeep], av[kDeep][RB];
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
          __builtin_memcpy(&xv[j], xrow + k + 32 * kSumWaves * j + lk, 16);
#pragma unroll
          for (int b = 0; b < RB; ++b) __builtin_memcpy(&av[j][b], arow[b] + k + 32 * kSumWaves * j + lk, 16);
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j)
#pragma unroll
          for (int b = 0; b < RB; ++b) acc[b] = M::mma(av[j][b], xv[j], acc[b]);
      }
      for (; k < k_end; k += 32 * kSumWaves) {
        const i32x4 xv = load_chunk(xrow, k + lk, k_end);
#pragma unroll
        for (int b = 0; b < RB; ++b) acc[b] = M::mma(load_chunk(arow[b], k + lk, k_end), xv, acc[b]);
      }
      __syncthreads();
#pragma unroll
      for (int b = 0; b < RB; ++b) sums[wave][b][lane] = acc[b];
      __syncthreads();
      // a thread has four rows of one block for one token
      for (int i = threadIdx.x; i < RB * 64; i += 64 * kSumWaves) {
        const int b = i / 64, l = i % 64, r = r0 + 16 * b + 4 * (l / 16);
        Acc s = sums[0][b][l];
#pragma unroll
        for (int w = 1; w < kSumWaves; ++w) s += sums[w][b][l];
        // (l is this thread's lane: 64 divides the step)
        if (own == adapter && r < pitch) {
          const float scale = ad.scale != nullptr ? ad.scale[adapter] : 1.0f;
          *reinterpret_cast<Acc*>(ad.s + (static_cast<long>(blockIdx.z) * rows + m0 + l % 16) * pitch + r) = s * scale;
        }
      }
    }
  }
}

// Few tokens: the depth is divided until there are about as many workgroups as CUs, into parts of
// at least 512.
int adapter_parts(long rows, long depth) {
  const long groups = (rows + 15) / 16 * std::min(rows, 16L);
  const long wanted = std::min({(256 + groups - 1) / std::max(groups, 1L), depth / 512, 16L});
  return static_cast<int>(std::max(wanted, 1L));
}

template <typename M, typename T>
static hipError_t adapter_sums(int rows, int depth, const void* x, long ldx, const Adapters& ad, hipStream_t st) {
  const int blocks = (rows + 15) / 16;
  // few tokens may have an adapter each; many, in long requests, mostly share one
  const dim3 grid(blocks, blocks <= 16 ? std::min(rows, 16) : 1, ad.parts);
  const int per = ((depth + ad.parts - 1) / ad.parts + 31) / 32 * 32;
  const auto kernel = ad.rank <= 16 ? adapter_sums_kernel<M, T, 1> : ad.rank <= 32 ? adapter_sums_kernel<M, T, 2> : adapter_sums_kernel<M, T, 4>;
  hipLaunchKernelGGL(kernel, grid, dim3(64 * kSumWaves), 0, st, rows, depth, per, static_cast<const T*>(x), ldx, ad);
  return hipGetLastError();
}

hipError_t launch_adapter_sums(int type, int rows, int depth, const void* x, long ldx, const Adapters& ad, hipStream_t st) {
  return type == kTypeBf16 ? adapter_sums<MmaBf16, bf16>(rows, depth, x, ldx, ad, st) : adapter_sums<MmaF16, f16>(rows, depth, x, ldx, ad, st);
}

}  // namespace oz2
