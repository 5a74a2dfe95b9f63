// oz2_adapters.hip -- S = scale X A^T, the first product of the adapters beside a linear layer.
#include <algorithm>
#include <cfloat>

#include "oz2_linear_tile.hpp"

namespace oz2 {

// ---- S as two 16-bit terms ----------------------------------------------------------------------
// The tile kernels' matrix instructions take S in 16 bits, while S is f32 in range and bits (it is
// scaled, and B may undo that): so it goes to them as the sum of two terms.  The first is S cut to the
// type's significant bits, and one unit of those less where it has no more, so that the second, the rest
// rounded, has its sign and is not zero: an infinite element of B then gives an infinity of the right
// sign, where zero times it, or the infinities of two signs, would make NaN.
//   bf16 (8 bits, f32's range): S is held within 2^-16 of itself.
//   f16 (11 bits): each 64 elements of a row have a unit, a power of two that puts their largest
// magnitude between 2^13 and 2^14, inside the range with as many bits below as there are; the sum with B is
// multiplied with it in f32.  S is held within 2^-22 of itself or 2^-37 of the largest.  (In f16 as it is, S
// past 65504 would be infinite, and below 2^-14 lose its bits.)
// One term of S costs less in the product, but the error of the result depends on it: with a residual
// that takes the leading bits away, one term's 2^-8 (bf16) is all that is left.  Both together cost 3% (bf16)
// and 5% (f16) of the prompts' product at rank 64.
__device__ __forceinline__ float finite_magnitude(float v) { return fabsf(v) <= FLT_MAX ? fabsf(v) : 0.0f; }

// What S is multiplied with, for the largest finite magnitude `top`, and the unit that undoes it (normal both).
template <typename T>
__device__ __forceinline__ float split_unit(float top, float& unit) {
  unit = 1.0f;
  if constexpr (std::is_same_v<T, bf16>) return 1.0f;
  const int n = min(14 - __builtin_amdgcn_frexp_expf(top), 113);
  unit = __builtin_amdgcn_ldexpf(1.0f, -n);
  return __builtin_amdgcn_ldexpf(1.0f, n);
}

template <typename T>
__device__ __forceinline__ void split_terms(float s, T& first, T& second) {
  first = static_cast<T>(s);
  second = static_cast<T>(0.0f);
  if (s == 0.0f || !(fabsf(s) <= FLT_MAX)) return;  // (an infinity less itself would be NaN)
  constexpr bool kHalf = std::is_same_v<T, f16>;
  const uint32_t cut = (__builtin_bit_cast(uint32_t, s) - 1) & (kHalf ? 0xFFFFE000u : 0xFFFF0000u);
  if (!kHalf || fabsf(s) >= 0x1p-13f) first = static_cast<T>(__builtin_bit_cast(float, cut));  // (exact)
  second = static_cast<T>(s - static_cast<float>(first));
  // (a rest below f16's subnormals)
  if (kHalf && second == static_cast<T>(0.0f)) second = static_cast<T>(__builtin_copysignf(0x1p-24f, s));
}

// 16 TB tokens and one of their adapters per workgroup, blockIdx.y the first of them that it takes (in
// the order of their first tokens) and blockIdx.z the part of the depth.  The matrix
// instruction's rows are 16 of the adapter's, its columns 16 tokens.  Operands go straight from
// memory to registers: a wave has a piece of the depth, in steps of 32 elements, DEEP of them
// under way.  Every token is computed and the adapter's own are stored.  RB: blocks of 16 rows of A
// that share the tokens' fragments; ranks above 64 take several passes.  SPLIT: the sums go out as split_terms
// has them.  Bound by what a CU draws from memory, some 40 GB/s: 8192 tokens of 24 requests at depth 2048, rank
// 64, 19.5 us (7 of them without any loads); 37 tokens with adapters of their own at depth 8192, rank 32, 8.0;
// one token at depth 2048, rank 16, 1.6.
template <typename M, typename T, bool SPLIT, int RB, int TB, int WAVES, int DEEP>
__global__ __launch_bounds__(64 * WAVES) void adapter_sums_kernel(int rows, int depth, int per, const T* __restrict__ x, long ldx,
                                                                  Adapters ad) {
  typedef typename M::acc Acc;
  constexpr int kTokens = 16 * TB;
  __shared__ Acc sums[WAVES][TB][RB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lk = 8 * (lane >> 4);
  const long m0 = static_cast<long>(kTokens) * blockIdx.x;
  const int own = lane < kTokens && m0 + lane < rows ? ad.index[m0 + lane] : -1;  // the adapter of the lane's token
  unsigned long todo = __ballot(own >= 0 && own < ad.count);
  const int pitch = ad.pitch();
  const int part_begin = per * static_cast<int>(blockIdx.z), part_end = min(part_begin + per, depth);
  const int steps = max(part_end - part_begin + 31, 0) / 32, each = (steps + WAVES - 1) / WAVES;
  const int k_begin = part_begin + 32 * each * wave, k_end = min(k_begin + 32 * each, part_end);
  const int whole = max(k_end - k_begin, 0) / 32;  // steps that the depth does not cut
  for (int n = 0; todo != 0; ++n) {
    const int token = __builtin_ctzl(todo), adapter = __builtin_amdgcn_readlane(own, token);
    const unsigned long match = __ballot(own == adapter);
    todo &= ~match;
    if (n % gridDim.y != blockIdx.y) continue;
    const float scale = ad.scale != nullptr ? ad.scale[adapter] : 1.0f;
    // a block without a token of the adapter's reads the first token's block again
    const T* xrow[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const int block = match >> (16 * t) & 0xFFFF ? t : token / 16;
      xrow[t] = x + min(m0 + 16 * block + li, static_cast<long>(rows) - 1) * ldx;
    }
    for (int r0 = 0; r0 < ad.rank; r0 += 16 * RB) {
      const T* arow[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b)
        arow[b] = static_cast<const T*>(ad.a) + adapter * ad.stride_a + min(r0 + 16 * b + li, ad.rank - 1) * ad.lda;
      Acc acc[TB][RB] = {};
      // N steps' loads under way together: without the fence the compiler puts each next to its use
      auto group = [&](int s, auto n) {
        constexpr int N = decltype(n)::value;
        i32x4 xv[N][TB], av[N][RB];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int k = k_begin + 32 * (s + j) + lk;
#pragma unroll
          for (int b = 0; b < RB; ++b) __builtin_memcpy(&av[j][b], arow[b] + k, 16);
#pragma unroll
          for (int t = 0; t < TB; ++t) __builtin_memcpy(&xv[j][t], xrow[t] + k, 16);
        }
        OZ2_SCHED_FENCE();
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int b = 0; b < RB; ++b) acc[t][b] = M::mma(av[j][b], xv[j][t], acc[t][b]);
      };
      int s = 0;
      for (; s + DEEP <= whole; s += DEEP) group(s, std::integral_constant<int, DEEP>{});
      for (; s + 2 <= whole; s += 2) group(s, std::integral_constant<int, 2>{});
      if (s < whole) group(s, std::integral_constant<int, 1>{});
      if (k_begin + 32 * whole < k_end) {
        const int k = k_begin + 32 * whole + lk;
        i32x4 av[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) av[b] = load_chunk(arow[b], k, k_end);
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          const i32x4 xv = load_chunk(xrow[t], k, k_end);
#pragma unroll
          for (int b = 0; b < RB; ++b) acc[t][b] = M::mma(av[b], xv, acc[t][b]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int b = 0; b < RB; ++b) sums[wave][t][b][lane] = acc[t][b];
      __syncthreads();
      if constexpr (SPLIT) {
        // a wave has all of a token's elements of this pass, whose largest sets their unit
        for (int t = wave; t < TB; t += WAVES) {
          float v[RB][4], top = 0.0f;
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            Acc s = sums[0][t][b][lane];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) s += sums[w][t][b][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[b][i] = r0 + 16 * b + lk / 2 + i < ad.rank ? s[i] * scale : 0.0f;
              top = fmaxf(top, finite_magnitude(v[b][i]));
            }
          }
          top = fmaxf(top, __shfl_xor(top, 16, 64));
          top = fmaxf(top, __shfl_xor(top, 32, 64));
          if ((match >> (16 * t + li) & 1) == 0) continue;
          const long m = m0 + 16 * t + li;
          float unit;
          const float per_unit = split_unit<T>(top, unit);
          if (std::is_same_v<T, f16> && lane < 16) ad.unit[m * ad.blocks() + r0 / 64] = unit;
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            const int r = r0 + 16 * b + lk / 2;
            if (r >= pitch) continue;
            T terms[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) split_terms(v[b][i] * per_unit, terms[0][i], terms[1][i]);
            char* const at = static_cast<char*>(ad.s) + 4 * (m * pitch + r / 8 * 8) + 2 * (r % 8);
            __builtin_memcpy(at, terms[0], sizeof(terms[0]));
            __builtin_memcpy(at + 16, terms[1], sizeof(terms[1]));
          }
        }
        continue;
      }
      // four rows of one block for one token each
      for (int i = threadIdx.x; i < TB * RB * 64; i += 64 * WAVES) {
        const int t = i / (64 * RB), b = i / 64 % RB, l = i % 64, r = r0 + 16 * b + 4 * (l / 16);
        if ((match >> (16 * t + l % 16) & 1) == 0 || r >= pitch) continue;
        Acc s = sums[0][t][b][l];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += sums[w][t][b][l];
#pragma unroll
        for (int v = 0; v < 4; ++v) s[v] = r + v < ad.rank ? s[v] * scale : 0.0f;
        const long m = m0 + 16 * t + l % 16;
        *reinterpret_cast<Acc*>(static_cast<float*>(ad.s) + (static_cast<long>(blockIdx.z) * rows + m) * pitch + r) = s;
      }
    }
  }
}

constexpr int kFewTokens = 256;  // rows up to which a workgroup takes 16 tokens and a part of the depth

// A CU draws some 40 GB/s from memory, so few rows are spread over the CUs by parts of the depth (37 rows
// with 32 adapters of rank 32 at depth 8192: 24 us in one part, 8.6 in 4, 7.0 in 16).  Dividing many made
// them no faster (8192 rows, rank 64, depth 2048: 19.6 us in one part and in two, 25 in four).  Between,
// a workgroup with 64 tokens and the whole depth takes as long as it does for 8192 rows, however few there are
// beside it, so there is a step behind the last of the few: 256 and 257 rows, rank 64, take 10 and 19 us at
// depth 2048 and 30 and 60 at depth 8192, rank 16 6 and 12, 14 and 38.
int adapter_parts(long rows, long depth) {
  return rows <= kFewTokens ? static_cast<int>(std::max(1L, std::min({depth / 512, 1024 / std::max(rows, 1L), 16L}))) : 1;
}

template <typename M, typename T>
static hipError_t adapter_sums(int rows, int depth, const void* x, long ldx, const Adapters& ad, hipStream_t st) {
  const int per = ((depth + ad.parts - 1) / ad.parts + 31) / 32 * 32;
  auto launch = [&](auto split, auto rb, auto tb, auto deep) {
    constexpr bool SPLIT = decltype(split)::value;
    constexpr int RB = decltype(rb)::value, TB = decltype(tb)::value, DEEP = decltype(deep)::value, kWaves = 4;
    const int groups = (rows + 16 * TB - 1) / (16 * TB);
    // workgroups that find no adapter left to them end at once
    const dim3 grid(groups, std::min({rows, 16 * TB, std::max(2, 1024 / groups)}), ad.parts);
    hipLaunchKernelGGL((adapter_sums_kernel<M, T, SPLIT, RB, TB, kWaves, DEEP>), grid, dim3(64 * kWaves), 0, st, rows, depth, per,
                       static_cast<const T*>(x), ldx, ad);
  };
  using std::integral_constant;
  auto ranks = [&](auto split, auto tb, auto deep) {
    if (ad.rank <= 16)
      launch(split, integral_constant<int, 1>{}, tb, integral_constant<int, 2 * decltype(deep)::value>{});
    else if (ad.rank <= 32)
      launch(split, integral_constant<int, 2>{}, tb, deep);
    else
      launch(split, integral_constant<int, 4>{}, tb, integral_constant<int, decltype(deep)::value / 2>{});
  };
  if (rows > kFewTokens)  // (one part, on tiles)
    ranks(std::true_type{}, integral_constant<int, 4>{}, integral_constant<int, 4>{});
  else if (ad.split && ad.parts == 1)
    ranks(std::true_type{}, integral_constant<int, 1>{}, integral_constant<int, 8>{});
  else
    ranks(std::false_type{}, integral_constant<int, 1>{}, integral_constant<int, 8>{});
  return hipGetLastError();
}

hipError_t launch_adapter_sums(int type, int rows, int depth, const void* x, long ldx, const Adapters& ad, hipStream_t st) {
  return type == kTypeBf16 ? adapter_sums<MmaBf16, bf16>(rows, depth, x, ldx, ad, st) : adapter_sums<MmaF16, f16>(rows, depth, x, ldx, ad, st);
}

// Adds up the parts of S and splits the sums, which take the place of the first part.  Sixteen threads of
// one wave for each 64 elements of a row, all of which are read before any is stored; eight parts' loads at a
// time.
template <typename T>
__global__ __launch_bounds__(64) void join_adapter_sums_kernel(int rows, Adapters ad) {
  const int at = static_cast<int>(threadIdx.x) & 15, pitch = ad.pitch();
  const long block = static_cast<long>(blockIdx.x) * 4 + threadIdx.x / 16, m = block / ad.blocks();
  const int k = 64 * static_cast<int>(block % ad.blocks()) + 4 * at;
  const bool own = m < rows && k < pitch;
  float* const s = static_cast<float*>(ad.s);
  const f32x4* const part = reinterpret_cast<const f32x4*>(s + (own ? m * pitch + k : 0));
  const long n = static_cast<long>(rows) * pitch / 4;
  f32x4 sum = {};
  for (int j = 0; j < ad.parts; j += 8) {
    f32x4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = part[min(j + u, ad.parts - 1) * n];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j + u < ad.parts) sum += v[u];
  }
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = fmaxf(top, own ? finite_magnitude(sum[i]) : 0.0f);
#pragma unroll
  for (int off = 1; off < 16; off *= 2) top = fmaxf(top, __shfl_xor(top, off, 64));
  if (!own) return;
  float unit;
  const float per_unit = split_unit<T>(top, unit);
  if (std::is_same_v<T, f16> && at == 0) ad.unit[block] = unit;
  T terms[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split_terms(sum[i] * per_unit, terms[0][i], terms[1][i]);
  char* const to = reinterpret_cast<char*>(s + m * pitch + k / 8 * 8) + 2 * (k % 8);
  __builtin_memcpy(to, terms[0], sizeof(terms[0]));
  __builtin_memcpy(to + 16, terms[1], sizeof(terms[1]));
}

hipError_t launch_join_adapter_sums(int type, int rows, const Adapters& ad, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>((static_cast<long>(rows) * ad.blocks() + 3) / 4));
  const auto kernel = type == kTypeBf16 ? join_adapter_sums_kernel<bf16> : join_adapter_sums_kernel<f16>;
  hipLaunchKernelGGL(kernel, grid, dim3(64), 0, st, rows, ad);
  return hipGetLastError();
}

// A thread per 16 bytes; blockIdx.y the adapter.  Every adapter's B is copied, used or not, by each call: 17 rows,
// 2048 -> 8192, rank 4 take 21.8 us with 8 adapters, 25.4 with 100 and 50 with 1000 (rank 8, whose B is read as
// it lies, 19.5 with any number).
__global__ __launch_bounds__(256) void pack_adapters_kernel(Adapters ad, int cols, uint16_t* dst) {
  const int per_row = packed_rank(ad.rank) / 8;
  const long n = static_cast<long>(blockIdx.x) * 256 + threadIdx.x, row = n / per_row;
  if (row >= cols) return;
  for (int a = blockIdx.y; a < ad.count; a += gridDim.y) {
    const uint16_t* const src = static_cast<const uint16_t*>(ad.b) + a * ad.stride_b + row * ad.ldb;
    const i32x4 v = load_chunk(src, 8 * static_cast<int>(n % per_row), ad.rank);
    *reinterpret_cast<i32x4*>(dst + 8 * (a * static_cast<long>(cols) * per_row + n)) = v;
  }
}

hipError_t launch_pack_adapters(const Adapters& ad, int cols, void* dst, hipStream_t st) {
  const long n = static_cast<long>(cols) * (packed_rank(ad.rank) / 8);
  const dim3 grid(static_cast<unsigned>((n + 255) / 256), std::min(ad.count, 32768));
  hipLaunchKernelGGL(pack_adapters_kernel, grid, dim3(256), 0, st, ad, cols, static_cast<uint16_t*>(dst));
  return hipGetLastError();
}

}  // namespace oz2
