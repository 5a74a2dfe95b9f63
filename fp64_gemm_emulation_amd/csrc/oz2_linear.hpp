// oz2_linear.hpp -- what the linear-layer kernels share: 16-bit element types, eight-element
// loads and stores, activations and their slopes, the counter-based dropout mask, and the
// epilogue that turns eight accumulators of one output row into stored results; and the host
// launch interface between oz2_linear_api.hip and the kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace oz2 {

typedef __bf16 bf16;
typedef _Float16 f16;

enum { kTypeBf16 = 0, kTypeF16 = 1, kTypeF32 = 2 };                            // mirror of oz2_type_t
enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };  // mirror of oz2_act_t

// Dropout as the kernels see it: keep where the 16-bit draw is at least t, times scale.
struct Drop {
  uint32_t t = 0;  // rint(2^16 p); 0: everything kept, 2^16: nothing
  // 2^16 / (2^16 - t), the reciprocal of the exact keep probability; with t = 0 in a gradient's
  // products, where nothing is dropped any more, the factor of their sums
  float scale = 1.0f;
  uint32_t k0 = 0, k1 = 0;  // key: the seed's halves
  uint32_t c2 = 0, c3 = 0;  // upper counter words: the offset's halves
};

// Epilogue of one product: out = res + drop(act(acc * xs[m] * ws[n] + bias[n])).
struct Epilogue {
  const void* bias = nullptr;  // [n], the operands' type
  int act = kActNone;
  Drop drop;
  const void* res = nullptr;  // residual, row stride ldr (may be y itself)
  long ldr = 0;
  void* z = nullptr;  // pre-activation output, row stride ldz
  long ldz = 0;
  void* y = nullptr;  // output, row stride ldy
  long ldy = 0;
  const float* xs = nullptr;  // int8 products: scale of each row of the left operand
  const float* ws = nullptr;  //               and of each row of the right one
};

// The power of two that a gradient's dZ is stored with.  Dropout's scale stays out of dZ (it
// multiplies the products' sums), so |dZ| is at most |dY| times the slope, and an activation's
// slope is at most 1.13: only there can f16 overflow, and half of dZ cannot.  It costs the last
// bit of values below 2^-13, and no rounding of others.
__host__ __device__ constexpr float dz_factor(bool f16, int act) { return f16 && act >= kActGelu ? 0.5f : 1.0f; }

// Which kernel computes a product, and over how many parts of the depth.
enum { kTile256 = 0, kTile128 = 1, kTile64 = 2, kFew8 = 3, kFew16 = 4, kTile128Deep = 5 };
struct Plan {
  int tile = kTile128;
  int splits = 1;
};
Plan plan_product(bool i8, long rows, long cols, long depth, bool left_along_index, bool right_along_index);
// Plans of dX (p x q, depth r) and dW (r x q, depth p); true: for launch_product_pair.
bool plan_pair(long p, long q, long r, Plan& dx, Plan& dw);
inline bool few_rows(const Plan& plan) { return plan.tile == kFew8 || plan.tile == kFew16; }
// Whether the workgroups of a product of few rows quantise them themselves: one or two rows,
// and at most 16 KB of levels.  Against a launch of its own before the product: 14.5 us and
// 18.5 for one row, 8192 x 8192 weights; 18.1 and 18.7 for two; four rows on 4096 x 4096
// weights are better quantised once, 10.1 us against 11.5.
inline bool quantize_in_product(const Plan& plan, long rows, long depth) {
  return few_rows(plan) && rows <= 2 && rows * ((depth + 15) / 16 * 16) <= 16384;
}
inline size_t partial_bytes(const Plan& plan, long rows, long cols) {
  return plan.splits > 1 ? 4 * static_cast<size_t>(plan.splits) * rows * ((cols + 7) / 8 * 8) : 0;
}

// Low-rank adapters beside a product, adapter a = index[m] of the row m (none outside 0 .. count - 1):
// the row's sum gets S_m B_a^T before the epilogue, S_m = scale_a X_m A_a^T.
struct Adapters {
  int count, rank;
  const void* a;  // [adapter][rank][depth], rows lda apart, adapters stride_a
  long lda, stride_a;
  const void* b;  // [adapter][cols][rank]
  long ldb, stride_b;
  const int32_t* index;
  const float* scale;  // null: ones
  // S, pitch() elements of four bytes to a row; rows without an adapter are not written.  `parts` sums over
  // parts of the depth, [part][row][pitch] in f32, as a product of few rows takes them, or, `split`, the whole
  // sums as two terms of the operands' type each, in the units of split_terms.
  void* s;
  int parts;
  bool split;
  float* unit;  // f16: of the 64 elements k of the row m at [m blocks() + k / 64]
  // (a product of more than a few rows reads B in pieces of 8 elements of rank: ranks between are packed)
  __host__ __device__ int pitch() const { return (rank + 15) / 16 * 16; }
  __host__ __device__ int blocks() const { return (rank + 63) / 64; }
};
// B with rows of ad.rank rounded up to a multiple of 8, zeros behind.
hipError_t launch_pack_adapters(const Adapters& ad, int cols, void* dst, hipStream_t st);
__host__ __device__ inline int packed_rank(int rank) { return (rank + 7) / 8 * 8; }
// Workgroups that share the depth of S.
int adapter_parts(long rows, long depth);
// The sum of ad's parts of S, split, in the place of the first part.
hipError_t launch_join_adapter_sums(int type, int rows, const Adapters& ad, hipStream_t st);
hipError_t launch_adapter_sums(int type, int rows, int depth, const void* x, long ldx, const Adapters& ad, hipStream_t st);

// out[m][n] = epilogue(sum_k left(m, k) right(n, k)), m < rows, n < cols, k < depth.  An operand
// lies along the depth (element (i, k) at i * ld + k) or along its index (at k * ld + i; products
// without an epilogue only).  Rows must be as rows_aligned says, except for
// kFew8 and kFew16.
struct Product {
  int type;   // element type of operands (unless int8) and outputs
  bool i8;    // int8 operands
  int rows, cols, depth;
  const void* left;
  long left_ld;
  bool left_along_index;
  const void* right;
  long right_ld;
  bool right_along_index;
  Epilogue epi;
  Plan plan;
  void* partial;  // partial_bytes of it
  bool quantize;  // int8 on kFew8 and kFew16: left is in the outputs' type, and is quantised by the kernel
};

// Whether the product kernels can take an operand as it lies: every row starts on a 16-byte
// boundary and is a multiple of 16 bytes long, and 256 rows stay within 32-bit offsets.
inline bool rows_aligned(const void* ptr, long ld, long len, int elem) {
  return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && ld * elem % 16 == 0 && len * elem % 16 == 0 &&
         ld * elem < (1L << 24);
}
// Row stride of a packed copy: a multiple of the cache line.
inline long packed_ld(long len, int elem) { return (len * elem + 127) / 128 * 128 / elem; }
struct PackJob {
  long rows;
  int cols;
  const void* src;
  long ld;
  void* dst;
  long ld_out;
};
// One or two operands (either may be null) in one launch.
hipError_t launch_pack_rows(int elem, const PackJob* a, const PackJob* b, hipStream_t st);

hipError_t launch_product(const Product& pr, hipStream_t st);
// With adapters, whose S is there: 16-bit operands along the depth.
hipError_t launch_product_adapters(const Product& pr, const Adapters& ad, hipStream_t st);
hipError_t launch_adapters_bf16(const Product& pr, const Adapters& ad, hipStream_t st);
hipError_t launch_adapters_f16(const Product& pr, const Adapters& ad, hipStream_t st);
// Sums of a gradient's dZ over its rows: db = scale times the sum over `blocks` partial rows of
// r floats (db null: none).
struct ColumnSums {
  int blocks, r;
  const float* part;
  float scale;
  void* db;
};
// Both products of a gradient and, where db is not null, the column sums, in one launch; the
// plans are plan_pair's.
hipError_t launch_product_pair(int type, const Product& dx, const Product& dw, const ColumnSums& sums, hipStream_t st);
hipError_t launch_pair_bf16(const Product& dx, const Product& dw, const ColumnSums& sums, hipStream_t st);
hipError_t launch_pair_f16(const Product& dx, const Product& dw, const ColumnSums& sums, hipStream_t st);
hipError_t launch_product_bf16(const Product& pr, hipStream_t st);
hipError_t launch_product_f16(const Product& pr, hipStream_t st);
hipError_t launch_product_i8(const Product& pr, hipStream_t st);
hipError_t launch_dropout_add(int type, int p, int r, const void* x, long ldx, const void* res, long ldr,
                              const Drop& drop, void* y, long ldy, hipStream_t st);
// dz = mask(dy) act'(z) dz_factor in the operands' type, mask being dropout without its scale
// (drop.scale is not used), its rows padded with zeros to a multiple of 8 (skipped when dz is
// null), and, when part is not null, the column sums of mask(dy) act'(z) over each of
// grad_row_blocks(p, r) blocks of rows: part is that many times r floats.  launch_column_sums
// adds them up.
int grad_row_blocks(int p, int r);
hipError_t launch_grad_rows(int type, int p, int r, const void* dy, long lddy, const void* z, long ldz, int act,
                            const Drop& drop, void* dz, long lddz, float* part, hipStream_t st);
hipError_t launch_column_sums(int type, const ColumnSums& sums, hipStream_t st);
// columns q .. fill - 1 of out are set to zero
hipError_t launch_quantize_rows(int type, int p, int q, const void* x, long ldx, int8_t* out, long ldo, int fill,
                                float* scale, hipStream_t st);

#ifdef __HIP_DEVICE_COMPILE__
#define OZ2_UNROLL _Pragma("unroll")
#else
#define OZ2_UNROLL
#endif

// f(activation) for the activation as a compile-time constant.
template <typename F>
__host__ __device__ __forceinline__ void with_activation(int act, F f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    default: f(std::integral_constant<int, kActNone>{}); break;
  }
}

// ---- eight consecutive elements ------------------------------------------------------
// Rows may start at any element, so these are unaligned vector accesses (the hardware's
// unaligned mode) where all eight lie inside the row, and single elements at its end.
// NT: with the non-temporal hint, for data that is read or written once and too large to be
// found in a cache later.
typedef int raw8 __attribute__((ext_vector_type(4)));  // eight 16-bit elements as they lie in memory
typedef raw8 raw8_unaligned __attribute__((aligned(2)));

template <bool NT>
__device__ __forceinline__ raw8 load16(const void* p) {
  if constexpr (NT) return __builtin_nontemporal_load(static_cast<const raw8_unaligned*>(p));
  raw8 r;
  __builtin_memcpy(&r, p, 16);
  return r;
}
template <bool NT>
__device__ __forceinline__ void store16(void* p, raw8 r) {
  if constexpr (NT) __builtin_nontemporal_store(r, static_cast<raw8_unaligned*>(p));
  else __builtin_memcpy(p, &r, 16);
}

template <typename T, bool NT = false>
__device__ __forceinline__ void load8(const T* p, int valid, float (&v)[8]) {
  T t[8];
  if (valid >= 8) {
    OZ2_UNROLL
    for (unsigned i = 0; i < sizeof(t) / 16; ++i) {
      const raw8 r = load16<NT>(reinterpret_cast<const char*>(p) + 16 * i);
      __builtin_memcpy(reinterpret_cast<char*>(t) + 16 * i, &r, 16);
    }
  } else {
    OZ2_UNROLL
    for (int i = 0; i < 8; ++i) t[i] = i < valid ? p[i] : static_cast<T>(0.0f);
  }
  OZ2_UNROLL
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(t[i]);
}

template <typename T, bool NT = false>
__device__ __forceinline__ void store8(T* p, int valid, const float (&v)[8]) {
  T t[8];
  OZ2_UNROLL
  for (int i = 0; i < 8; ++i) t[i] = static_cast<T>(v[i]);
  if (valid >= 8) {
    OZ2_UNROLL
    for (unsigned i = 0; i < sizeof(t) / 16; ++i) {
      raw8 r;
      __builtin_memcpy(&r, reinterpret_cast<const char*>(t) + 16 * i, 16);
      store16<NT>(reinterpret_cast<char*>(p) + 16 * i, r);
    }
  } else {
    OZ2_UNROLL
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = t[i];
  }
}

// ---- activations -----------------------------------------------------------------------
// gelu(a) = a Phi(a), Phi the normal distribution function; gelu_tanh is its tanh form,
// a sigmoid(2 c (a + k a^3)) with c = sqrt(2 / pi), k = 0.044715; silu(a) = a sigmoid(a).
// In a product's epilogue these are work that the matrix cores wait for, so they are built
// from the hardware's exponential and reciprocal (each within 2^-23, relative).
__device__ __forceinline__ float exp_fast(float v) { return __builtin_amdgcn_exp2f(v * 1.4426950408889634f); }
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + exp_fast(-v)); }
__device__ __forceinline__ float sigmoid_gelu_tanh(float a) {
  return sigmoid(a * __builtin_fmaf(1.5957691216057308f * 0.044715f, a * a, 1.5957691216057308f));
}

// Phi(-|a|) = erfc(|a| / sqrt 2) / 2 from a and e = exp(-a^2 / 2), by formula 7.1.26 of Abramowitz and
// Stegun, "Handbook of Mathematical Functions" (a fifth-degree polynomial in
// 1 / (1 + 0.3275911 x) times exp(-x^2), within 1.5e-7): a third of the instructions of erff.
__device__ __forceinline__ float normal_tail(float a, float e) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f * 0.70710678118654752f, fabsf(a), 1.0f));
  float p = __builtin_fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f);
  p = __builtin_fmaf(t, p, 0.5f * 1.421413741f);
  p = __builtin_fmaf(t, p, 0.5f * -0.284496736f);
  p = __builtin_fmaf(t, p, 0.5f * 0.254829592f);
  return t * p * e;
}

template <int ACT>
__device__ __forceinline__ float activate(float a) {
  if constexpr (ACT == kActRelu) {
    return a <= 0.0f ? 0.0f : a;  // NaN stays NaN
  } else if constexpr (ACT == kActGelu) {
    // max(a, 0) - |a| Phi(-|a|); the minimum keeps +Inf from meeting its factor 0
    const float h = normal_tail(a, exp_fast(-0.5f * a * a));
    return __builtin_fmaf(-fabsf(fminf(a, 65536.0f)), h, fmaxf(a, 0.0f));
  } else if constexpr (ACT == kActGeluTanh) {
    return a * sigmoid_gelu_tanh(a);
  } else if constexpr (ACT == kActSilu) {
    return a * sigmoid(a);
  } else {
    return a;
  }
}

// The slopes have reached their limits (0 and 1, in f32) well before |z| = 100.  Beyond, the
// formulas would multiply 0 by infinity (z^2 past 1.8e19, or an infinite z, as a pre-activation
// past f16's range is kept), so their outer z is held within 1e4; NaN comes through s or h.
template <int ACT>
__device__ __forceinline__ float activation_slope(float z) {
  const float zc = __builtin_amdgcn_fmed3f(z, -1e4f, 1e4f);
  if constexpr (ACT == kActRelu) {
    return z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActGelu) {
    const float e = __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);  // a multiply less than exp_fast
    const float h = normal_tail(z, e);
    return __builtin_fmaf(zc * 0.39894228040143268f, e, z > 0.0f ? 1.0f - h : h);
  } else if constexpr (ACT == kActGeluTanh) {
    const float s = sigmoid_gelu_tanh(z);
    return s + zc * s * (1.0f - s) * 1.5957691216057308f * __builtin_fmaf(3.0f * 0.044715f, zc * zc, 1.0f);
  } else if constexpr (ACT == kActSilu) {
    const float s = sigmoid(z);
    return s * (1.0f + zc * (1.0f - s));
  } else {
    return 1.0f;
  }
}

// ---- dropout -----------------------------------------------------------------------------
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// 2011).  One block serves eight consecutive elements of one row, 16 bits each: the keep
// probability is then a multiple of 2^-16, and its exact value sets the scale, so the
// expectation is exact; two blocks of 32-bit draws would double the generator's cost (20
// full-width multiplies at a quarter of the vector rate per block), which the matrix cores wait
// for in an epilogue (in dropout_add the memory's time covers it).
__host__ __device__ __forceinline__ void philox_block(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
  // a loop: unrolled into every eight outputs of an epilogue, the rounds alone outgrow the
  // instruction cache
#pragma unroll 1
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(c[0]) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c[2]) * 0xCD9E8D57u;
    const uint32_t n0 = static_cast<uint32_t>(b >> 32) ^ c[1] ^ k0;
    const uint32_t n2 = static_cast<uint32_t>(a >> 32) ^ c[3] ^ k1;
    c[0] = n0;
    c[1] = static_cast<uint32_t>(b);
    c[2] = n2;
    c[3] = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// v[i] <- element 8 block8 + i of its row, dropped or scaled (SCALE false: dropped or left).  A
// dropped element is 0 whatever it held (Inf and NaN too).
template <bool SCALE = true>
__device__ __forceinline__ void drop8(float (&v)[8], const Drop& d, long row, int cols, int block8) {
  const uint64_t n = static_cast<uint64_t>(row) * static_cast<uint64_t>((cols + 7) >> 3) + static_cast<uint64_t>(block8);
  uint32_t c[4] = {static_cast<uint32_t>(n), static_cast<uint32_t>(n >> 32), d.c2, d.c3};
  philox_block(c, d.k0, d.k1);
  OZ2_UNROLL
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = (i & 1) ? c[i >> 1] >> 16 : c[i >> 1] & 0xFFFFu;
    v[i] = u >= d.t ? (SCALE ? v[i] * d.scale : v[i]) : 0.0f;
  }
}

// ---- quantisation ----------------------------------------------------------------------------
constexpr float kTinyRow = 1e-36f;

// Largest magnitude of eight values; +Inf if one is NaN.
__device__ __forceinline__ float magnitude8(const float (&v)[8]) {
  float top = 0.0f;
  OZ2_UNROLL
  for (int i = 0; i < 8; ++i) top = v[i] != v[i] ? __builtin_inff() : fmaxf(top, fabsf(v[i]));
  return top;
}

__device__ __forceinline__ float wave_max_magnitude(float top) {
  OZ2_UNROLL
  for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  return top;
}

// The factor 127 / top that a row's elements are multiplied with, and its scale `step`.
__device__ __forceinline__ float quantization(float top, float& step) {
  const bool finite = top <= 3.4028234e38f, live = finite && top >= kTinyRow;
  step = live ? top / 127.0f : finite ? 0.0f : __builtin_nanf("");
  return live ? 127.0f / top : 0.0f;
}

// The level of one element (0 in a row without a finite scale).
__device__ __forceinline__ int level(float v, float inv) { return inv != 0.0f ? static_cast<int>(rintf(v * inv)) : 0; }

// Levels of v[0 .. valid) to p, zeros behind them up to `count` (at most 8).
__device__ __forceinline__ void store_levels(int8_t* p, int count, int valid, const float (&v)[8], float inv) {
  int8_t t[8];
  OZ2_UNROLL
  for (int i = 0; i < 8; ++i) t[i] = static_cast<int8_t>(i < valid ? level(v[i], inv) : 0);
  if (count >= 8) {
    __builtin_memcpy(p, t, 8);
  } else {
    OZ2_UNROLL
    for (int i = 0; i < 8; ++i)
      if (i < count) p[i] = t[i];
  }
}

// ---- epilogue ------------------------------------------------------------------------------
// What an epilogue reads for eight columns, as it lies in memory.
template <typename T, bool FULL, bool NT = false>
__device__ __forceinline__ raw8 load_raw8(const void* base, long at, int valid) {
  const T* const p = static_cast<const T*>(base) + at;
  if (FULL || valid >= 8) return load16<NT>(p);
  T t[8];
  OZ2_UNROLL
  for (int i = 0; i < 8; ++i) t[i] = i < valid ? p[i] : static_cast<T>(0.0f);
  raw8 r;
  __builtin_memcpy(&r, t, sizeof(r));
  return r;
}

template <typename T>
__device__ __forceinline__ float raw_element(const raw8& r, int i) {
  T t[8];
  __builtin_memcpy(t, &r, sizeof(r));
  return static_cast<float>(t[i]);
}

// Eight accumulators of row m, columns n .. n + 7 (n a multiple of 8, n < cols), with the
// operands of the epilogue already read (those that the Epilogue names).  FULL: the columns
// are a multiple of 8, so no group is cut (a quarter of the code).
template <typename T, int ACT, bool FULL, bool NT = false>
__device__ __forceinline__ void finish8(float (&v)[8], const Epilogue& e, long m, int n, int cols, float xs,
                                        const float (&ws)[8], const raw8& bias, const raw8& res) {
  const int valid = FULL ? 8 : cols - n;
  if (e.xs != nullptr) {
    OZ2_UNROLL
    for (int i = 0; i < 8; ++i) v[i] = v[i] * xs * ws[i];
  }
  if (e.bias != nullptr) {
    OZ2_UNROLL
    for (int i = 0; i < 8; ++i) v[i] += raw_element<T>(bias, i);
  }
  if (e.z != nullptr) store8<T, NT>(static_cast<T*>(e.z) + m * e.ldz + n, valid, v);
  if constexpr (ACT != kActNone) {
    OZ2_UNROLL
    for (int i = 0; i < 8; ++i) v[i] = activate<ACT>(v[i]);
  }
  if (e.drop.t != 0) drop8(v, e.drop, m, cols, n >> 3);
  if (e.res != nullptr) {
    OZ2_UNROLL
    for (int i = 0; i < 8; ++i) v[i] += raw_element<T>(res, i);
  }
  store8<T, NT>(static_cast<T*>(e.y) + m * e.ldy + n, valid, v);
}

// The same for one group by itself.
template <typename T, int ACT, bool FULL>
__device__ __forceinline__ void finish8(float (&v)[8], const Epilogue& e, long m, int n, int cols) {
  const int valid = FULL ? 8 : cols - n;
  float xs = 0.0f, ws[8] = {};
  raw8 bias = {}, res = {};
  if (e.res != nullptr) res = load_raw8<T, FULL>(e.res, m * e.ldr + n, valid);
  if (e.bias != nullptr) bias = load_raw8<T, FULL>(e.bias, n, valid);
  if (e.xs != nullptr) {
    xs = e.xs[m];
    load8(e.ws + n, valid, ws);
  }
  finish8<T, ACT, FULL>(v, e, m, n, cols, xs, ws, bias, res);
}

// ---- column sums ---------------------------------------------------------------------------
// ColumnSums, kSumColumns columns per workgroup of THREADS threads, in a fixed order; lds:
// THREADS floats.
constexpr int kSumColumns = 32;

template <typename T, int THREADS>
__device__ __forceinline__ void column_sums(float* lds, unsigned wg, const ColumnSums& sums) {
  constexpr int W = THREADS / kSumColumns;
  const int lane = threadIdx.x % kSumColumns, w = threadIdx.x / kSumColumns;
  const int c = static_cast<int>(wg) * kSumColumns + lane;
  float s = 0.0f;
  if (c < sums.r) {
#pragma unroll 4
    for (int b = w; b < sums.blocks; b += W) s += sums.part[static_cast<long>(b) * sums.r + c];
  }
  lds[threadIdx.x] = s;
  __syncthreads();
  if (w != 0 || c >= sums.r) return;
  s = 0.0f;
  OZ2_UNROLL
  for (int i = 0; i < W; ++i) s += lds[i * kSumColumns + lane];
  static_cast<T*>(sums.db)[c] = static_cast<T>(s * sums.scale);
}

}  // namespace oz2
