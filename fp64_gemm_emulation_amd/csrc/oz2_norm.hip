// oz2_norm.hip -- the root-mean-square norm around the linear-layer products, with the residual's
// addition and int8 rows, and its gradient.
#include <algorithm>

#include "oz2_common.hpp"
#include "oz2_linear.hpp"
#include "oz2_norm.hpp"

namespace oz2 {

// Matrices above this are read and written with the non-temporal hint: with their like they
// exceed the 256 MB memory-side cache.
constexpr double kStreamBytes = 64.0 * (1 << 20);

// Eight elements as they lie in memory.
template <typename T>
struct Raw {
  raw8 r[sizeof(T) / 2];
};

template <typename T, bool NT>
__device__ __forceinline__ Raw<T> load_raw(const T* p, int valid) {
  Raw<T> o;
  if (valid >= 8) {
    OZ2_UNROLL
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) o.r[i] = load16<NT>(reinterpret_cast<const char*>(p) + 16 * i);
  } else {
    T t[8];
    OZ2_UNROLL
    for (int i = 0; i < 8; ++i) t[i] = i < valid ? p[i] : static_cast<T>(0.0f);
    __builtin_memcpy(&o, t, sizeof(o));
  }
  return o;
}

template <typename T>
__device__ __forceinline__ void widen(const Raw<T>& o, float (&v)[8]) {
  T t[8];
  __builtin_memcpy(t, &o, sizeof(o));
  OZ2_UNROLL
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(t[i]);
}

__device__ __forceinline__ float wave_sum(float v) {
  OZ2_UNROLL
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Reductions over the THREADS threads of a row, in a fixed order; slots: one value per wave.
template <int THREADS>
__device__ __forceinline__ float row_sum(float v, float* slots) {
  v = wave_sum(v);
  if constexpr (THREADS > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
    OZ2_UNROLL
    for (int i = 0; i < THREADS / 64; ++i) v += slots[i];
  }
  return v;
}
template <int THREADS>
__device__ __forceinline__ float row_max(float v, float* slots) {
  v = wave_max_magnitude(v);
  if constexpr (THREADS > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
    OZ2_UNROLL
    for (int i = 0; i < THREADS / 64; ++i) v = fmaxf(v, slots[i]);
  }
  return v;
}

// A row's values are multiplied with `pre` and then with `rstd`.  Squares of bf16 and f32 values
// may pass f32's range although the norm does not: where their sum has, the row's values go through
// 2^-80 first (2^128 then squares to 2^96, and 2^15 of them add up to 2^111; eps is far below).
constexpr float kSmall = 0x1p-80f;
template <int THREADS, int HELD>
__device__ __forceinline__ void norm_factors(const float (&v)[HELD][8], float sum, int q, float eps, float* slots,
                                             float& pre, float& rstd) {
  pre = 1.0f;
  if (!(sum <= 3.0e38f)) {  // uniform over the row's threads
    pre = kSmall;
    float s = 0.0f;
    OZ2_UNROLL
    for (int c = 0; c < HELD; ++c)
      OZ2_UNROLL
      for (int i = 0; i < 8; ++i) s = __builtin_fmaf(v[c][i] * kSmall, v[c][i] * kSmall, s);
    sum = row_sum<THREADS>(s, slots);
    eps = 0.0f;
  }
  rstd = 1.0f / __builtin_sqrtf(sum / static_cast<float>(q) + eps);
}

// One row per THREADS threads (several rows to a workgroup of 256 where a wave holds one), HELD
// groups of eight elements per thread, so a row is read once and stays in registers between its
// sum, its products and, for int8, its largest magnitude.  Bound by memory: 16384 x 8192 bf16 with a
// residual in 174 us, 6.2 TB/s (157 with int8 rows); one row of 8192 in 4.4 us in a trace, mostly the launch and
// two trips through LDS.  f32: 8192 x 8192 in 222 us, 4.8 TB/s, 2048 x 2048 14.2.  Rows above 8192, by 1024 threads:
// 8192 x 16384 bf16 in 196 us (240 with int8 rows), f32 425 (403); 256 x 32768 bf16 14.4.
template <typename T, int THREADS, int HELD, bool I8, bool NT>
__global__ __launch_bounds__(THREADS < 256 ? 256 : THREADS) void rms_norm_kernel(Norm n) {
  constexpr int kGroup = THREADS < 256 ? 256 : THREADS, kRows = kGroup / THREADS;
  __shared__ float slots[kGroup / 64];
  const int t = threadIdx.x % THREADS;
  const T* const w = static_cast<const T*>(n.w);
  for (long row = static_cast<long>(blockIdx.x) * kRows + threadIdx.x / THREADS; row < n.p; row += static_cast<long>(gridDim.x) * kRows) {
    const T* const x = static_cast<const T*>(n.x) + row * n.ldx;
    const T* const res = n.res != nullptr ? static_cast<const T*>(n.res) + row * n.ldr : nullptr;
    T* const h = n.h != nullptr ? static_cast<T*>(n.h) + row * n.ldh : nullptr;
    Raw<T> xr[HELD] = {}, rr[HELD] = {};
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
      const int k = 8 * (t + THREADS * c);
      if (k >= n.q) continue;
      xr[c] = load_raw<T, NT>(x + k, n.q - k);
      if (res != nullptr) rr[c] = load_raw<T, NT>(res + k, n.q - k);
    }
    float v[HELD][8], sum = 0.0f;
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
      const int k = 8 * (t + THREADS * c);
      widen(xr[c], v[c]);
      if (res != nullptr) {
        float r[8];
        widen(rr[c], r);
        // rounded as it is stored: the norm is of what the stream carries on
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = static_cast<float>(static_cast<T>(v[c][i] + r[i]));
      }
      if (h != nullptr && k < n.q) store8<T, NT>(h + k, n.q - k, v[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(v[c][i], v[c][i], sum);
    }
    sum = row_sum<THREADS>(sum, slots);
    float pre, rstd;
    norm_factors<THREADS, HELD>(v, sum, n.q, n.eps, slots, pre, rstd);
    float top = 0.0f;
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
      const int k = 8 * (t + THREADS * c);
      if (k >= n.q) continue;
      float g[8];
      if (w != nullptr) load8(w + k, n.q - k, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * pre * rstd * (w != nullptr ? g[i] : 1.0f);
      if constexpr (I8) {
        // (beyond the row's end a NaN or an infinite rstd has made NaN of zeros)
        float m[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = k + i < n.q ? v[c][i] : 0.0f;
        top = fmaxf(top, magnitude8(m));
      } else {
        store8<T, NT>(static_cast<T*>(n.y) + row * n.ldy + k, n.q - k, v[c]);
      }
    }
    if constexpr (I8) {
      top = row_max<THREADS>(top, slots);
      float step;
      const float inv = quantization(top, step);
#pragma unroll
      for (int c = 0; c < HELD; ++c) {
        const int k = 8 * (t + THREADS * c);
        if (k < n.q) store_levels(n.levels + row * n.ldl + k, n.q - k, n.q - k, v[c], inv);
      }
      if (t == 0) n.scale[row] = step;
    }
  }
}

template <typename T, bool I8>
static hipError_t rms_norm(const Norm& n, hipStream_t st) {
  const bool nt = static_cast<double>(n.p) * n.q * sizeof(T) > kStreamBytes;
  const int groups = (n.q + 7) / 8;
  auto launch = [&](auto threads, auto held) {
    constexpr int THREADS = decltype(threads)::value, HELD = decltype(held)::value;
    constexpr int kGroup = THREADS < 256 ? 256 : THREADS, kRows = kGroup / THREADS;
    const dim3 grid(static_cast<unsigned>(std::min((static_cast<long>(n.p) + kRows - 1) / kRows, 1L << 20)));
    const auto kernel = nt ? rms_norm_kernel<T, THREADS, HELD, I8, true> : rms_norm_kernel<T, THREADS, HELD, I8, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(kGroup), 0, st, n);
  };
  // As few threads as hold the row without idle ones, and for few long rows twice as many.  Times of
  // 64 x 4, 256 x 1 and 512 x 2 threads x groups: 16384 x 512 15.3 (64 x 1: 13.2), 20.9 and 50 us; 777 x
  // 1999 6.4, 5.5 and 7.1; 65536 x 1024 88 (64 x 2: 88), 102 and 226; 16384 x 2048 41.8, 41.4 and 56.
  // Of 256 x 4, 512 x 2 and 1024 x 1: 64 x 8192 5.1, 4.1 and 4.3; 2048 x 8192 22.9, 22.0 and 24.2; 16384 x
  // 8192 174, 175 and 174, with int8 rows 157, 159 and 265.
  using std::integral_constant;
  if (groups <= 64)
    launch(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (groups <= 128)
    launch(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (groups <= 256)
    launch(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (groups <= 1024 && n.p <= 2048)
    launch(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  else if (groups <= 1024)
    launch(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  else
    launch(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
  return hipGetLastError();
}

hipError_t launch_rms_norm(const Norm& n, hipStream_t st) {
  const bool i8 = n.y == nullptr;
  if (n.type == kTypeBf16) return i8 ? rms_norm<bf16, true>(n, st) : rms_norm<bf16, false>(n, st);
  if (n.type == kTypeF16) return i8 ? rms_norm<f16, true>(n, st) : rms_norm<f16, false>(n, st);
  return i8 ? rms_norm<float, true>(n, st) : rms_norm<float, false>(n, st);
}

// ---- gradient ------------------------------------------------------------------------------
// With n = h rstd and g = dy w: dx = rstd (g - n mean(g n)) + dh, dw = the sum of dy n over rows.
// Both sums of a row come from one pass, as mean(g n) = rstd mean(g h); so the forward call leaves
// nothing but h.  A workgroup takes every gridDim-th row (rows), and adds up its part of dw in
// registers.  Bound by memory: 16384 x 8192 bf16 with dh in 177 us, 6.1 TB/s; f32 8192 x 8192, with the sums
// of dw's parts, 211.  Rows above 8192 are not: 1024 threads have 128 registers each, which w, dw, h and dy of 32
// columns outgrow, and 472 to 484 bytes of scratch memory a lane hold the rest: 8192 x 16384 820 us (f32 1185), 4096 x
// 32768 684, 256 x 16384 52.
template <typename T, int THREADS, int HELD, bool NT>
__global__ __launch_bounds__(THREADS < 256 ? 256 : THREADS) void rms_norm_bwd_kernel(NormGrad n) {
  constexpr int kGroup = THREADS < 256 ? 256 : THREADS, kRows = kGroup / THREADS;
  __shared__ float slots[kGroup / 64];
  const int t = threadIdx.x % THREADS;
  const float count = static_cast<float>(n.q);
  float w[HELD][8], dw[HELD][8] = {};
#pragma unroll
  for (int c = 0; c < HELD; ++c) {
    const int k = 8 * (t + THREADS * c);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[c][i] = 1.0f;
    if (n.w != nullptr && k < n.q) load8(static_cast<const T*>(n.w) + k, n.q - k, w[c]);
  }
  for (long row = static_cast<long>(blockIdx.x) * kRows + threadIdx.x / THREADS; row < n.p; row += static_cast<long>(gridDim.x) * kRows) {
    const T* const hp = static_cast<const T*>(n.h) + row * n.ldh;
    const T* const dyp = static_cast<const T*>(n.dy) + row * n.lddy;
    const T* const dhp = n.dh != nullptr ? static_cast<const T*>(n.dh) + row * n.lddh : nullptr;
    Raw<T> hr[HELD] = {}, gr[HELD] = {}, ar[HELD] = {};
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
      const int k = 8 * (t + THREADS * c);
      if (k >= n.q) continue;
      hr[c] = load_raw<T, NT>(hp + k, n.q - k);
      gr[c] = load_raw<T, NT>(dyp + k, n.q - k);
      if (dhp != nullptr) ar[c] = load_raw<T, NT>(dhp + k, n.q - k);
    }
    float h[HELD][8], squares = 0.0f, mixed = 0.0f;
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
      float g[8];
      widen(hr[c], h[c]);
      widen(gr[c], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        squares = __builtin_fmaf(h[c][i], h[c][i], squares);
        mixed = __builtin_fmaf(g[i] * w[c][i], h[c][i], mixed);
      }
    }
    squares = row_sum<THREADS>(squares, slots);
    mixed = row_sum<THREADS>(mixed, slots);
    float pre, rstd;
    norm_factors<THREADS, HELD>(h, squares, n.q, n.eps, slots, pre, rstd);
    float mean = mixed / count * rstd;  // of g n
    if (!(squares <= 3.0e38f && fabsf(mixed) <= 3.0e38f)) {
      mixed = 0.0f;
#pragma unroll
      for (int c = 0; c < HELD; ++c) {
        float g[8];
        widen(gr[c], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) mixed = __builtin_fmaf(g[i] * w[c][i], h[c][i] * pre * rstd, mixed);
      }
      mean = row_sum<THREADS>(mixed, slots) / count;
    }
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
      const int k = 8 * (t + THREADS * c);
      if (k >= n.q) continue;
      float g[8], a[8], d[8];
      widen(gr[c], g);
      widen(ar[c], a);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float norm = h[c][i] * pre * rstd;
        d[i] = __builtin_fmaf(__builtin_fmaf(-norm, mean, g[i] * w[c][i]), pre * rstd, a[i]);
        dw[c][i] = __builtin_fmaf(g[i], norm, dw[c][i]);
      }
      if (n.dx != nullptr) store8<T, NT>(static_cast<T*>(n.dx) + row * n.lddx + k, n.q - k, d);
    }
  }
  if (n.dw == nullptr) return;
  float* const part = n.part + static_cast<long>(blockIdx.x) * n.q;
  if constexpr (kRows > 1) {
    __shared__ float sums[kRows][THREADS][8];
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[threadIdx.x / THREADS][t][i] = dw[c][i];
      __syncthreads();
      for (int j = threadIdx.x; j < 8 * THREADS; j += kGroup) {
        const int k = 8 * THREADS * c + j;
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) s += sums[r][j / 8][j % 8];
        if (k < n.q) part[k] = s;
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
      const int k = 8 * (t + THREADS * c);
      if (k < n.q) store8(part + k, n.q - k, dw[c]);
    }
  }
}

// f(threads per row, groups of eight they hold, most workgroups), by the matrix's size.  More
// workgroups mean shorter loops over rows and more partial sums of dw.  Times without the sums of the
// parts: of 64 x 4 and 256 x 1 threads x groups, 256 x 2048 6.4 and 4.0 us, 16384 x 2048 45 and 58 (512
// workgroups); of 256 x 4 and 512 x 2, 256 x 8192 8.0 and 7.2, 512 x 8192 11.6 and 10.3 (256
// workgroups), 16384 x 8192 177 and 210 (512; 228 and 206 with 256).
template <typename F>
static void with_grad_row(int p, int q, F f) {
  using std::integral_constant;
  const int groups = (q + 7) / 8;
  if (groups <= 128)
    f(integral_constant<int, 64>{}, integral_constant<int, 2>{}, 512);
  else if (groups <= 256 && p <= 1024)
    f(integral_constant<int, 256>{}, integral_constant<int, 1>{}, 512);
  else if (groups <= 256)
    f(integral_constant<int, 64>{}, integral_constant<int, 4>{}, 512);
  else if (groups <= 1024 && p <= 512)
    f(integral_constant<int, 512>{}, integral_constant<int, 2>{}, 256);
  else if (groups <= 1024)
    f(integral_constant<int, 256>{}, integral_constant<int, 4>{}, 512);
  else
    f(integral_constant<int, 1024>{}, integral_constant<int, 4>{}, 512);
}

int norm_grad_blocks(int p, int q) {
  int blocks = 0;
  with_grad_row(p, q, [&](auto threads, auto, int most) {
    constexpr int THREADS = decltype(threads)::value, kRows = THREADS < 256 ? 256 / THREADS : 1;
    blocks = std::min((p + kRows - 1) / kRows, most);
  });
  return blocks;
}

template <typename T>
static hipError_t rms_norm_bwd(const NormGrad& n, hipStream_t st) {
  const bool nt = static_cast<double>(n.p) * n.q * sizeof(T) > kStreamBytes;
  const int blocks = norm_grad_blocks(n.p, n.q);
  if (blocks > 0) {
    with_grad_row(n.p, n.q, [&](auto threads, auto held, int) {
      constexpr int THREADS = decltype(threads)::value, HELD = decltype(held)::value;
      const auto kernel = nt ? rms_norm_bwd_kernel<T, THREADS, HELD, true> : rms_norm_bwd_kernel<T, THREADS, HELD, false>;
      hipLaunchKernelGGL(kernel, dim3(blocks), dim3(THREADS < 256 ? 256 : THREADS), 0, st, n);
    });
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (n.dw == nullptr) return hipSuccess;
  return launch_column_sums(n.type, ColumnSums{blocks, n.q, n.part, 1.0f, n.dw}, st);
}

hipError_t launch_rms_norm_bwd(const NormGrad& n, hipStream_t st) {
  if (n.type == kTypeBf16) return rms_norm_bwd<bf16>(n, st);
  return n.type == kTypeF16 ? rms_norm_bwd<f16>(n, st) : rms_norm_bwd<float>(n, st);
}

}  // namespace oz2
