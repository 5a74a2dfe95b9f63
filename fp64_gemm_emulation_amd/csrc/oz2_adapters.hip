// oz2_adapters.hip -- S = scale X A^T, the first product of the adapters beside a linear layer.
#include <algorithm>

#include "oz2_linear_tile.hpp"

namespace oz2 {

// 16 TB tokens and one of their adapters per workgroup, blockIdx.y the first of them that it takes (in
// the order of their first tokens) and blockIdx.z the part of the depth.  The matrix
// instruction's rows are 16 of the adapter's, its columns 16 tokens.  Operands go straight from
// memory to registers: a wave has a piece of the depth, in steps of 32 elements, DEEP of them
// under way.  Every token is computed and the adapter's own are stored.  RB: blocks of 16 rows of A
// that share the tokens' fragments; ranks above 64 take several passes.  Bound by what a CU draws from
// memory, some 40 GB/s: 8192 tokens of 24 requests at depth 2048, rank 64, 19.1 us (7 of them without
// any loads); 37 tokens with adapters of their own at depth 8192, rank 32, 7.8; one token at depth 2048, rank
// 16, 1.7.
template <typename M, typename T, int RB, int TB, int WAVES, int DEEP>
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
        if (ad.rounded) {
          T half[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) half[v] = static_cast<T>(s[v]);
          __builtin_memcpy(static_cast<T*>(ad.s) + m * pitch + r, half, sizeof(half));
        } else {
          *reinterpret_cast<Acc*>(static_cast<float*>(ad.s) + (static_cast<long>(blockIdx.z) * rows + m) * pitch + r) = s;
        }
      }
    }
  }
}

constexpr int kFewTokens = 256;  // rows up to which a workgroup takes 16 tokens and a part of the depth

// A CU draws some 40 GB/s from memory, so few rows are spread over the CUs by parts of the depth (37 rows
// with 32 adapters of rank 32 at depth 8192: 24 us in one part, 8.6 in 4, 7.0 in 16).  Many have
// workgroups enough; dividing those made them no faster (8192 rows, rank 64, depth 2048: 19.6 us in one
// part and in two, 25 in four).
int adapter_parts(long rows, long depth) {
  return rows <= kFewTokens ? static_cast<int>(std::max(1L, std::min({depth / 512, 1024 / std::max(rows, 1L), 16L}))) : 1;
}

template <typename M, typename T>
static hipError_t adapter_sums(int rows, int depth, const void* x, long ldx, const Adapters& ad, hipStream_t st) {
  const int per = ((depth + ad.parts - 1) / ad.parts + 31) / 32 * 32;
  auto launch = [&](auto rb, auto tb, auto deep) {
    constexpr int RB = decltype(rb)::value, TB = decltype(tb)::value, DEEP = decltype(deep)::value, kWaves = 4;
    const int groups = (rows + 16 * TB - 1) / (16 * TB);
    // workgroups that find no adapter left to them end at once
    const dim3 grid(groups, std::min({rows, 16 * TB, std::max(2, 1024 / groups)}), ad.parts);
    hipLaunchKernelGGL((adapter_sums_kernel<M, T, RB, TB, kWaves, DEEP>), grid, dim3(64 * kWaves), 0, st, rows, depth, per,
                       static_cast<const T*>(x), ldx, ad);
  };
  using std::integral_constant;
  auto ranks = [&](auto tb, auto deep) {
    if (ad.rank <= 16)
      launch(integral_constant<int, 1>{}, tb, integral_constant<int, 2 * decltype(deep)::value>{});
    else if (ad.rank <= 32)
      launch(integral_constant<int, 2>{}, tb, deep);
    else
      launch(integral_constant<int, 4>{}, tb, integral_constant<int, decltype(deep)::value / 2>{});
  };
  if (rows <= kFewTokens)
    ranks(integral_constant<int, 1>{}, integral_constant<int, 8>{});
  else
    ranks(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  return hipGetLastError();
}

hipError_t launch_adapter_sums(int type, int rows, int depth, const void* x, long ldx, const Adapters& ad, hipStream_t st) {
  return type == kTypeBf16 ? adapter_sums<MmaBf16, bf16>(rows, depth, x, ldx, ad, st) : adapter_sums<MmaF16, f16>(rows, depth, x, ldx, ad, st);
}

// Adds up the parts of S, rounded: four elements per thread, four parts' loads at a time.
template <typename T>
__global__ __launch_bounds__(64) void join_adapter_sums_kernel(long n, int parts, const f32x4* __restrict__ s, T* __restrict__ out) {
  const long at = static_cast<long>(blockIdx.x) * 64 + threadIdx.x;
  if (at >= n) return;
  f32x4 sum = {};
  for (int j = 0; j < parts; j += 4) {
    f32x4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = s[min(j + u, parts - 1) * n + at];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (j + u < parts) sum += v[u];
  }
  T t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = static_cast<T>(sum[i]);
  __builtin_memcpy(out + 4 * at, t, sizeof(t));
}

hipError_t launch_join_adapter_sums(int type, int rows, const Adapters& ad, void* out, hipStream_t st) {
  const long n = static_cast<long>(rows) * ad.pitch() / 4;
  const dim3 grid(static_cast<unsigned>((n + 63) / 64));
  const f32x4* const s = static_cast<const f32x4*>(ad.s);
  if (type == kTypeBf16)
    hipLaunchKernelGGL(join_adapter_sums_kernel<bf16>, grid, dim3(64), 0, st, n, ad.parts, s, static_cast<bf16*>(out));
  else
    hipLaunchKernelGGL(join_adapter_sums_kernel<f16>, grid, dim3(64), 0, st, n, ad.parts, s, static_cast<f16*>(out));
  return hipGetLastError();
}

// A thread per 16 bytes; blockIdx.y the adapter.
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
