// oz2_linear_rows.hip -- the row-wise passes around the linear-layer products: dropout with
// residual, the gradient before the products with its column sums, and the quantisation of
// rows to int8.
#include "oz2_common.hpp"
#include "oz2_linear.hpp"

namespace oz2 {

// Matrices above this are read and written with the non-temporal hint: with their like they
// exceed the 256 MB memory-side cache.
constexpr double kStreamBytes = 64.0 * (1 << 20);

// y = res + drop(x): one thread per eight consecutive elements of a row, so one generator
// block per thread.  Bound by memory: 16384 x 8192 bf16 with a residual in 127 us, 6.3 TB/s
// (174 us without the non-temporal hint); vector instructions issue in 65% of the cycles
// meanwhile.  A workgroup covers cx column groups (a power of two) of 256 / cx rows.
template <typename T, bool NT>
__global__ __launch_bounds__(256) void dropout_add_kernel(int p, int r, int cx_log2, const T* x, long ldx, const T* res,
                                                          long ldr, Drop d, T* y, long ldy) {
  const int b = (blockIdx.x << cx_log2) + (threadIdx.x & ((1 << cx_log2) - 1));
  const int valid = r - 8 * b;
  if (valid <= 0) return;
  const int ry = 256 >> cx_log2;
  for (long row = static_cast<long>(blockIdx.y) * ry + (threadIdx.x >> cx_log2); row < p;
       row += static_cast<long>(gridDim.y) * ry) {
    float v[8], t[8];
    load8<T, NT>(x + row * ldx + 8 * b, valid, v);
    if (d.t != 0) drop8(v, d, row, r, b);
    if (res != nullptr) {
      load8<T, NT>(res + row * ldr + 8 * b, valid, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += t[i];
    }
    store8<T, NT>(y + row * ldy + 8 * b, valid, v);
  }
}

template <typename T>
static hipError_t dropout_add(int p, int r, const void* x, long ldx, const void* res, long ldr, const Drop& d, void* y,
                              long ldy, hipStream_t st) {
  const int groups = (r + 7) >> 3;
  int cx_log2 = 0;
  while (cx_log2 < 8 && (1 << cx_log2) < groups) ++cx_log2;
  const int ry = 256 >> cx_log2;
  const long row_blocks = (static_cast<long>(p) + ry - 1) / ry;
  const dim3 grid((groups + (1 << cx_log2) - 1) >> cx_log2, static_cast<unsigned>(row_blocks < 65535 ? row_blocks : 65535));
  const auto kernel = static_cast<double>(p) * r * sizeof(T) > kStreamBytes ? dropout_add_kernel<T, true> : dropout_add_kernel<T, false>;
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, p, r, cx_log2, static_cast<const T*>(x), ldx,
                     static_cast<const T*>(res), ldr, d, static_cast<T*>(y), ldy);
  return hipGetLastError();
}

hipError_t launch_dropout_add(int type, int p, int r, const void* x, long ldx, const void* res, long ldr,
                              const Drop& drop, void* y, long ldy, hipStream_t st) {
  if (type == kTypeBf16) return dropout_add<bf16>(p, r, x, ldx, res, ldr, drop, y, ldy, st);
  if (type == kTypeF16) return dropout_add<f16>(p, r, x, ldx, res, ldr, drop, y, ldy, st);
  return dropout_add<float>(p, r, x, ldx, res, ldr, drop, y, ldy, st);
}

// dz = mask(dy) act'(z) dz_factor: a workgroup takes a block of rows of 256 columns, a thread eight
// consecutive columns of every eighth row.  Column sums are of the unrounded f32 values, in
// a fixed order: over the thread's rows, over the eight threads of a column group, and (in
// column_sums_kernel) over the row blocks.  Bound by memory: 8192 x 8192 bf16, gelu, in 77 us,
// 5.2 TB/s.
constexpr int kGradCols = 256;

// Rows per block: as many, up to 256, as leave 1024 workgroups (four per CU), for fewer
// partial sums; at least 16.
static int grad_block_rows(int p, int r) {
  const long col_blocks = (static_cast<long>(r) + kGradCols - 1) / kGradCols;
  int rows = 256;
  while (rows > 16 && (p + rows - 1) / rows * col_blocks < 1024) rows /= 2;
  return rows;
}

int grad_row_blocks(int p, int r) {
  const int rows = grad_block_rows(p, r);
  return (p + rows - 1) / rows;
}

template <typename T, int ACT>
__global__ __launch_bounds__(256) void grad_rows_kernel(int p, int r, const T* dy, long lddy, const T* z, long ldz,
                                                        Drop d, T* dz, long lddz, int block_rows, float* part) {
  __shared__ float sums[8][kGradCols];
  const int g = threadIdx.x & 31, rr = threadIdx.x >> 5;
  const int col = blockIdx.y * kGradCols + 8 * g;
  const int valid = r - col;
  const long row0 = static_cast<long>(blockIdx.x) * block_rows;
  float sum[8] = {};
  if (valid > 0) {
    for (long row = row0 + rr; row < min(row0 + block_rows, static_cast<long>(p)); row += 8) {
      float v[8], t[8];
      load8<T, true>(dy + row * lddy + col, valid, v);
      if (d.t != 0) drop8<false>(v, d, row, r, col >> 3);
      if constexpr (ACT != kActNone) {
        load8<T, true>(z + row * ldz + col, valid, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= activation_slope<ACT>(t[i]);
      }
      // dz's rows are padded to multiples of 8 with zeros (load8's)
      if (dz != nullptr) {
        constexpr float kFactor = dz_factor(std::is_same_v<T, f16>, ACT);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = v[i] * kFactor;
        store8(dz + row * lddz + col, 8, t);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[i];
    }
  }
  if (part == nullptr) return;  // uniform over the launch
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[rr][8 * g + i] = sum[i];
  __syncthreads();
  const int c = blockIdx.y * kGradCols + threadIdx.x;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += sums[i][threadIdx.x];
  if (c < r) part[static_cast<long>(blockIdx.x) * r + c] = s;
}

template <typename T>
__global__ __launch_bounds__(256) void column_sums_kernel(ColumnSums sums) {
  __shared__ float lds[256];
  column_sums<T, 256>(lds, blockIdx.x, sums);
}

hipError_t launch_column_sums(int type, const ColumnSums& sums, hipStream_t st) {
  const auto kernel = type == kTypeBf16 ? column_sums_kernel<bf16> : type == kTypeF16 ? column_sums_kernel<f16> : column_sums_kernel<float>;
  hipLaunchKernelGGL(kernel, dim3((sums.r + kSumColumns - 1) / kSumColumns), dim3(256), 0, st, sums);
  return hipGetLastError();
}

template <typename T>
static hipError_t grad_rows(int p, int r, const void* dy, long lddy, const void* z, long ldz, int act, const Drop& d,
                            void* dz, long lddz, float* part, hipStream_t st) {
  if (p == 0 || r == 0) return hipSuccess;
  const dim3 grid(grad_row_blocks(p, r), (r + kGradCols - 1) / kGradCols);
  with_activation(act, [&](auto a) {
    hipLaunchKernelGGL((grad_rows_kernel<T, decltype(a)::value>), grid, dim3(256), 0, st, p, r, static_cast<const T*>(dy),
                       lddy, static_cast<const T*>(z), ldz, d, static_cast<T*>(dz), lddz, grad_block_rows(p, r), part);
  });
  return hipGetLastError();
}

hipError_t launch_grad_rows(int type, int p, int r, const void* dy, long lddy, const void* z, long ldz, int act,
                            const Drop& drop, void* dz, long lddz, float* part, hipStream_t st) {
  if (type == kTypeBf16) return grad_rows<bf16>(p, r, dy, lddy, z, ldz, act, drop, dz, lddz, part, st);
  return grad_rows<f16>(p, r, dy, lddy, z, ldz, act, drop, dz, lddz, part, st);
}

// Row quantisation: scale = max|x| / 127, q = rint(x (127 / max|x|)); a row whose
// largest magnitude is below kTinyRow (127 / it would overflow) is taken for zeros, with scale
// 0, and one that holds Inf or NaN gets the scale NaN, so its products are NaN.  One
// workgroup per row, eight elements per thread at a time; the first kHeld of them stay in
// registers between the two passes, so rows up to 8192 are read once.  8192 x 2048 bf16 in
// 14.6 us, 3.4 TB/s with the launch in it.
constexpr int kHeld = 4;

template <typename T>
__global__ __launch_bounds__(256) void quantize_rows_kernel(int q, const T* x, long ldx, int8_t* out, long ldo, int fill,
                                                            float* scale) {
  __shared__ float tops[4];
  const long row = blockIdx.x;
  const T* const src = x + row * ldx;
  int8_t* const dst = out + row * ldo;
  float held[kHeld][8], v[8];
  float top = 0.0f;
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int k = 8 * (threadIdx.x + 256 * h);
    if (k < q) {
      load8(src + k, q - k, held[h]);
      top = fmaxf(top, magnitude8(held[h]));
    }
  }
  for (int k = 8 * (threadIdx.x + 256 * kHeld); k < q; k += 8 * 256) {
    load8(src + k, q - k, v);
    top = fmaxf(top, magnitude8(v));
  }
  top = wave_max_magnitude(top);
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  float step;
  const float inv = quantization(top, step);
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int k = 8 * (threadIdx.x + 256 * h);
    if (k < fill) store_levels(dst + k, min(fill - k, 8), q - k, held[h], inv);
  }
  for (int k = 8 * (threadIdx.x + 256 * kHeld); k < fill; k += 8 * 256) {
    if (k < q) load8(src + k, q - k, v);
    store_levels(dst + k, min(fill - k, 8), q - k, v, inv);
  }
  if (threadIdx.x == 0) scale[row] = step;
}

hipError_t launch_quantize_rows(int type, int p, int q, const void* x, long ldx, int8_t* out, long ldo, int fill,
                                float* scale, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(p));
  if (type == kTypeBf16)
    hipLaunchKernelGGL(quantize_rows_kernel<bf16>, grid, dim3(256), 0, st, q, static_cast<const bf16*>(x), ldx, out, ldo, fill, scale);
  else if (type == kTypeF16)
    hipLaunchKernelGGL(quantize_rows_kernel<f16>, grid, dim3(256), 0, st, q, static_cast<const f16*>(x), ldx, out, ldo, fill, scale);
  else
    hipLaunchKernelGGL(quantize_rows_kernel<float>, grid, dim3(256), 0, st, q, static_cast<const float*>(x), ldx, out, ldo, fill, scale);
  return hipGetLastError();
}

}  // namespace oz2
