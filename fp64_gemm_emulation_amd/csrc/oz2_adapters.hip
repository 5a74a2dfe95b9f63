// oz2_adapters.hip -- S = scale X A^T, the first product of the adapters beside a linear layer.
#include <algorithm>

#include "oz2_linear_tile.hpp"

namespace oz2 {

// 16 TB tokens and one of their adapters per workgroup, blockIdx.y the first of them that it
// takes (in the order of their first tokens) and blockIdx.z the part of the depth.  The matrix
// instruction's rows are 16 of the adapter's, its columns 16 tokens.  Operands go straight from
// memory to registers: a wave has a block of tokens and a contiguous piece of the depth, in steps
// of 32 elements, kDeep of them under way; the pieces start at different memory channels (rows a
// power of two apart would otherwise all ask the same one).  Every column is computed and the
// adapter's own tokens are stored.  RB: blocks of 16 rows that share the tokens' fragments; ranks above
// 64 take several passes.
constexpr int kSumWaves = 16;

template <typename M, typename T, int RB, int TB>
__global__ __launch_bounds__(64 * kSumWaves) void adapter_sums_kernel(int rows, int depth, int per, const T* __restrict__ x,
                                                                      long ldx, Adapters ad) {
  typedef typename M::acc Acc;
  constexpr int kDeep = RB == 4 ? 2 : 4, kPieces = kSumWaves / TB;
  __shared__ Acc sums[kPieces][TB][RB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int block = wave % TB, piece = wave / TB;
  const int li = lane & 15, lk = 8 * (lane >> 4);
  const long m0 = 16l * TB * blockIdx.x;
  // the adapter of the lane's token, and the tokens that are the first of theirs
  int own = lane < 16 * TB && m0 + lane < rows ? ad.index[m0 + lane] : -1;
  if (own >= ad.count) own = -1;
  bool first = own >= 0;
#pragma unroll
  for (int j = 0; j < 16 * TB - 1; ++j) {
    const int before = __builtin_amdgcn_readlane(own, j);
    first = first && (j >= lane || before != own);
  }
  unsigned long firsts = __ballot(first);
  const int part_begin = per * static_cast<int>(blockIdx.z), part_end = min(part_begin + per, depth);
  const int steps = max(part_end - part_begin + 31, 0) / 32, each = (steps + kPieces - 1) / kPieces;
  const int k_begin = part_begin + 32 * each * piece, k_end = min(k_begin + 32 * each, part_end);
  const T* const xrow = x + min(m0 + 16 * block + li, static_cast<long>(rows) - 1) * ldx;
  const int pitch = ad.pitch();
  for (int n = 0; firsts != 0; ++n) {
    const int token = __builtin_ctzl(firsts);
    firsts &= firsts - 1;
    if (n % gridDim.y != blockIdx.y) continue;
    const int adapter = __builtin_amdgcn_readlane(own, token);
    const unsigned long match = __ballot(own == adapter);
    for (int r0 = 0; r0 < ad.rank; r0 += 16 * RB) {
      const T* arow[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b)
        arow[b] = static_cast<const T*>(ad.a) + adapter * ad.stride_a + min(r0 + 16 * b + li, ad.rank - 1) * ad.lda;
      Acc acc[RB] = {};
      if (match >> (16 * block) & 0xFFFF) {
        int k = k_begin;
        for (; k + 32 * kDeep <= k_end; k += 32 * kDeep) {
          i32x4 xv[kDeep], av[kDeep][RB];
#pragma unroll
          for (int j = 0; j < kDeep; ++j) {
            __builtin_memcpy(&xv[j], xrow + k + 32 * j + lk, 16);
#pragma unroll
            for (int b = 0; b < RB; ++b) __builtin_memcpy(&av[j][b], arow[b] + k + 32 * j + lk, 16);
          }
#pragma unroll
          for (int j = 0; j < kDeep; ++j)
#pragma unroll
            for (int b = 0; b < RB; ++b) acc[b] = M::mma(av[j][b], xv[j], acc[b]);
        }
        for (; k < k_end; k += 32) {
          const i32x4 xv = load_chunk(xrow, k + lk, k_end);
          i32x4 av[RB];
#pragma unroll
          for (int b = 0; b < RB; ++b) av[b] = load_chunk(arow[b], k + lk, k_end);
#pragma unroll
          for (int b = 0; b < RB; ++b) acc[b] = M::mma(av[b], xv, acc[b]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int b = 0; b < RB; ++b) sums[piece][block][b][lane] = acc[b];
      __syncthreads();
      // four rows of one block for one token each
      for (int i = threadIdx.x; i < TB * RB * 64; i += 64 * kSumWaves) {
        const int t = i / (64 * RB), b = i / 64 % RB, l = i % 64, r = r0 + 16 * b + 4 * (l / 16);
        if ((match >> (16 * t + l % 16) & 1) == 0 || r >= pitch) continue;
        Acc s = sums[0][t][b][l];
#pragma unroll
        for (int w = 1; w < kPieces; ++w) s += sums[w][t][b][l];
        s *= ad.scale != nullptr ? ad.scale[adapter] : 1.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (r + v >= ad.rank) s[v] = 0.0f;
        *reinterpret_cast<Acc*>(ad.s + (static_cast<long>(blockIdx.z) * rows + m0 + 16 * t + l % 16) * pitch + r) = s;
      }
    }
  }
}

// Few tokens: the depth is divided until there are about as many workgroups as CUs, into parts of
// at least 512.
int adapter_parts(long rows, long depth) {
  const long groups = rows <= 256 ? (rows + 15) / 16 * std::min(rows, 16L) : (rows + 31) / 32;
  const long wanted = std::min({(256 + groups - 1) / std::max(groups, 1L), depth / 512, 16L});
  return static_cast<int>(std::max(wanted, 1L));
}

template <typename M, typename T>
static hipError_t adapter_sums(int rows, int depth, const void* x, long ldx, const Adapters& ad, hipStream_t st) {
  const int per = ((depth + ad.parts - 1) / ad.parts + 31) / 32 * 32;
  auto launch = [&](auto ranks, auto tokens) {
    constexpr int RB = decltype(ranks)::value, TB = decltype(tokens)::value;
    // few tokens may have an adapter each; many, in long requests, mostly share one
    const dim3 grid((rows + 16 * TB - 1) / (16 * TB), TB == 1 ? std::min(rows, 16) : 1, ad.parts);
    hipLaunchKernelGGL((adapter_sums_kernel<M, T, RB, TB>), grid, dim3(64 * kSumWaves), 0, st, rows, depth, per,
                       static_cast<const T*>(x), ldx, ad);
  };
  auto blocks = [&](auto ranks) {
    rows <= 256 ? launch(ranks, std::integral_constant<int, 1>{}) : launch(ranks, std::integral_constant<int, 2>{});
  };
  if (ad.rank <= 16)
    blocks(std::integral_constant<int, 1>{});
  else if (ad.rank <= 32)
    blocks(std::integral_constant<int, 2>{});
  else
    blocks(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

hipError_t launch_adapter_sums(int type, int rows, int depth, const void* x, long ldx, const Adapters& ad, hipStream_t st) {
  return type == kTypeBf16 ? adapter_sums<MmaBf16, bf16>(rows, depth, x, ldx, ad, st) : adapter_sums<MmaF16, f16>(rows, depth, x, ldx, ad, st);
}

}  // namespace oz2
