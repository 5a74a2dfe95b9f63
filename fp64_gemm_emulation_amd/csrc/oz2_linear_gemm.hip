// oz2_linear_gemm.hip -- out = epilogue(left right^T), the products of the linear layer and of
// its gradient: bf16 and f16 operands with f32 accumulators, int8 operands with int32 ones
// (exact: 127^2 times the depth stays below 2^31 up to the 2^17 the entry points accept).
#include <type_traits>

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

#define OZ2_WAIT_VMCNT(N) __builtin_amdgcn_s_waitcnt(((N) & 0xF) | (((N) >> 4) << 14) | (0x7 << 4) | (0xF << 8))
#define OZ2_WAIT_LGKMCNT(N) __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4) | (((N) & 0xF) << 8))
#define OZ2_SCHED_FENCE() __builtin_amdgcn_sched_barrier(0)

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef short s16x4 __attribute__((ext_vector_type(4)));

// What the tile kernel does with its accumulators.
enum { kOutEpilogue = 0, kOutPlain = 1 };

// 256 x 256 tiles from this many of them on (one per CU); 128 x 128 tiles below.
constexpr long kBigTiles = 256;

// How an operand lies in memory: along the depth (element (i, k) at i * ld + k), or along its
// own index (at k * ld + i), as W does in dX = dZ W and both operands do in dW = dZ^T X.
enum { kAlongDepth = 0, kAlongIndex = 1 };

// ---- tile kernel ---------------------------------------------------------------------
// BT x BT outputs per workgroup (BT = 256: 8 waves in 2 x 4, two to a SIMD, 128 x 64 outputs
// each; BT = 128: 4 waves in 2 x 2, 64 x 64 each, two workgroups to a CU).  Depth advances in
// stages of 128 bytes, so that every row of an operand along the depth brings whole cache
// lines; two stages are held in LDS, filled with 1 KiB copies straight from memory.
//
// Per stage and wave, two halves of 64 bytes of depth (one matrix instruction deep):
//   first half:  MFMAs on the first fragments, the second half's fragments read between them;
//   middle:      every wave has read the stage: wait for the copies of the next stage (issued
//                one stage ago), barrier;
//   second half: MFMAs on the second fragments, between them the copies of the stage after
//                next into the buffer just released, and the next stage's first fragments.
// So there is one barrier per stage, and a copy has a whole stage of MFMAs to arrive.
//
// LDS layouts and bank conflicts.  Along the depth: rows of 128 bytes, 16-byte chunk c of row
// i at chunk c ^ s(i).  The 16 lanes that read one chunk of 16 rows then hit 16 different
// 16-byte bank groups (64 banks of 4 bytes): rows alternate between the halves of the banks
// by their lowest bit, and s takes 8 values over those with the same one.  The right operand's
// rows are dealt to the fragments so that a lane ends up with eight consecutive output
// columns (block b of a pair takes rows 8 g + 4 b + v of 32, g = 0..3, v = 0..3), and its s is
// chosen for that set.  Along the index: depth rows of BT elements, 32-byte block c of row k
// at block c ^ f(k), read with the transposing LDS read: 16 lanes fetch 4 depth rows x 16
// indices, each lane 8 bytes, and each receives one index's 4 depths.  f takes 16 (BT = 256)
// or, within either half of the wave, 8 (BT = 128) values over the 16 rows one read touches.
template <int BT>
struct Tile {
  static constexpr int WAVES = BT == 256 ? 8 : 4;
  static constexpr int WN = BT == 256 ? 4 : 2;  // waves along the columns, the other two along the rows
  static constexpr int MB = BT / 32;            // 16-row blocks per wave
  static constexpr int NB = BT / (16 * WN);     // 16-column blocks per wave
  static constexpr int SLICE = BT * 128;        // bytes of one operand's stage
  static constexpr int COPIES = SLICE / 1024 / WAVES;  // per wave and operand (4)
};

// s(i) of an operand along the depth.
template <bool RIGHT>
__device__ __forceinline__ int chunk_swizzle(int i) {
  return RIGHT ? (((i >> 3) & 3) << 1) | ((i >> 1) & 1) : (i >> 1) & 7;
}
// f(k) of an operand along the index.
template <int BT>
__device__ __forceinline__ int block_swizzle(int k) {
  return (k & 3) | (((k >> 3) & (BT == 256 ? 3 : 1)) << 2);
}

// Byte offset, from the operand's tile origin, of the 16 bytes that lane `lane` copies with
// the 1 KiB unit u of a stage; `tail`: what to add in the last stage so that chunks beyond
// the depth read something inside the row (they are zeroed in LDS afterwards).
template <int BT, int E, int LAYOUT, bool RIGHT>
__device__ __forceinline__ unsigned copy_offset(int u, int lane, long ld, int last_index, int last_stage_depth, int* tail) {
  if constexpr (LAYOUT == kAlongDepth) {
    const int i = 8 * u + (lane >> 3);
    const int c = (lane & 7) ^ chunk_swizzle<RIGHT>(i);
    *tail = c * (16 / E) < last_stage_depth ? 0 : -16 * c;
    return static_cast<unsigned>(min(i, last_index) * static_cast<unsigned>(ld) * E + 16 * c);
  } else {
    constexpr int kRow = BT * E, kPerRow = kRow / 16;  // bytes and 16-byte chunks of a depth row
    const int k = u * (1024 / kRow) + lane / kPerRow;
    const int pc = lane % kPerRow;
    const int c = 2 * ((pc >> 1) ^ block_swizzle<BT>(k)) + (pc & 1);
    *tail = k < last_stage_depth ? 0 : static_cast<int>((last_stage_depth - 1 - k) * ld * E);
    // columns beyond the last chunk only reach outputs that are not stored
    return static_cast<unsigned>(k * static_cast<unsigned>(ld) * E + min(16 * c, last_index / (16 / E) * 16));
  }
}

__device__ __forceinline__ void tile_of(unsigned wg, int tiles_m, int tiles_n, int& ti, int& tj) {
  // workgroups go round-robin over the 8 XCDs: give each XCD a contiguous range of tiles, and
  // walk it in groups of 4 tile rows, so the workgroups on one XCD's L2 share operand panels
  constexpr unsigned kXcds = 8, kGroup = 4;
  const unsigned n = static_cast<unsigned>(tiles_m) * static_cast<unsigned>(tiles_n);
  const unsigned x = wg % kXcds, per = n / kXcds, rem = n % kXcds;
  const unsigned id = x * per + min(x, rem) + wg / kXcds;
  const unsigned group = id / (kGroup * tiles_n), in_group = id % (kGroup * tiles_n);
  const unsigned rows = min(static_cast<unsigned>(tiles_m) - group * kGroup, kGroup);
  ti = static_cast<int>(group * kGroup + in_group % rows);
  tj = static_cast<int>(in_group / rows);
}

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

// The transposing read of 8 bytes per lane.  A function with a restrict pointer, so that the
// load carries aliasing information: without any, the compiler makes it wait for every copy
// into LDS that is still in flight.
__device__ __forceinline__ s16x4 read_transposed(__attribute__((address_space(3))) s16x4* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}

template <typename M, typename T, int BT, int LL, int RL, int OUT>
__global__ __launch_bounds__(64 * Tile<BT>::WAVES, BT == 256 ? 1 : 2) void product_tile_kernel(
    int rows, int cols, int depth, const typename M::elem* __restrict__ left, long left_ld,
    const typename M::elem* __restrict__ right, long right_ld, Epilogue e, int tiles_m, int tiles_n) {
  typedef Tile<BT> S;
  typedef typename M::acc Acc;
  constexpr int E = sizeof(typename M::elem);
  constexpr int kDepth = 128 / E;  // elements of depth per stage
  constexpr int MB = S::MB, NB = S::NB, FR = MB + NB, COPIES = S::COPIES;
  __shared__ __attribute__((aligned(1024))) char smem[2 * 2 * S::SLICE];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // waves w and w + 4 share a SIMD: the same rows, so the left fragments repeat there
  const int wm = wave & 1, wn = wave >> 1;
  int ti, tj;
  tile_of(blockIdx.x, tiles_m, tiles_n, ti, tj);
  const long m0 = static_cast<long>(ti) * BT;
  const int n0 = tj * BT;

  const int nk = (depth + kDepth - 1) / kDepth;
  const int last_depth = depth - (nk - 1) * kDepth;  // elements of depth in the last stage
  const char* const lbase = reinterpret_cast<const char*>(left) + (LL == kAlongDepth ? m0 * left_ld : m0) * E;
  const char* const rbase = reinterpret_cast<const char*>(right) + (RL == kAlongDepth ? n0 * right_ld : n0) * E;
  const long lstep = LL == kAlongDepth ? 128 : kDepth * left_ld * E;
  const long rstep = RL == kAlongDepth ? 128 : kDepth * right_ld * E;
  const int last_m = static_cast<int>(min(static_cast<long>(rows) - 1 - m0, static_cast<long>(BT - 1)));
  const int last_n = min(cols - 1 - n0, BT - 1);
  unsigned loff[COPIES], roff[COPIES];
  int ltail[COPIES], rtail[COPIES];
#pragma unroll
  for (int j = 0; j < COPIES; ++j) {
    loff[j] = copy_offset<BT, E, LL, false>(wave + S::WAVES * j, lane, left_ld, last_m, last_depth, &ltail[j]);
    roff[j] = copy_offset<BT, E, RL, true>(wave + S::WAVES * j, lane, right_ld, last_n, last_depth, &rtail[j]);
  }
  // copy j (the left operand's first) of stage kt into its buffer
  auto copy1 = [&](int kt, int j) {
    char* const dst = smem + (kt & 1) * 2 * S::SLICE + (wave + S::WAVES * (j % COPIES)) * 1024;
    const bool last = kt == nk - 1;
    if (j < COPIES)
      __builtin_amdgcn_global_load_lds(
          static_cast<const void*>(lbase + kt * lstep + (loff[j % COPIES] + (last ? ltail[j % COPIES] : 0))), (lds_ptr_t)dst, 16, 0, 0);
    else
      __builtin_amdgcn_global_load_lds(
          static_cast<const void*>(rbase + kt * rstep + (roff[j % COPIES] + (last ? rtail[j % COPIES] : 0))),
          (lds_ptr_t)(dst + S::SLICE), 16, 0, 0);
  };
  // zeroes what lies beyond the depth in the last stage's buffer
  auto clear_tail = [&]() {
    char* const buf = smem + ((nk - 1) & 1) * 2 * S::SLICE;
    for (int n = tid; n < 2 * S::SLICE / 16; n += 64 * S::WAVES) {
      const bool r = n >= S::SLICE / 16;
      const int c = r ? n - S::SLICE / 16 : n;
      bool beyond;
      if ((r ? RL : LL) == kAlongDepth)
        beyond = ((c & 7) ^ (r ? chunk_swizzle<true>(c >> 3) : chunk_swizzle<false>(c >> 3))) * (16 / E) >= last_depth;
      else
        beyond = c / (BT * E / 16) >= last_depth;
      if (beyond) *reinterpret_cast<i32x4*>(buf + 16 * n) = i32x4{0, 0, 0, 0};
    }
  };

  // fragment reads
  const int li = lane & 15, lg = lane >> 4;
  int la[LL == kAlongDepth ? 1 : MB], ra[RL == kAlongDepth ? 1 : NB];
  if constexpr (LL == kAlongDepth) {
    const int i = wm * (16 * MB) + li;
    la[0] = 128 * i + 16 * (lg ^ chunk_swizzle<false>(i));
  } else {
    const int k = 8 * lg + (li >> 2);
#pragma unroll
    for (int b = 0; b < MB; ++b) la[b] = BT * E * k + 32 * ((wm * MB + b) ^ block_swizzle<BT>(k)) + 8 * (li & 3);
  }
  if constexpr (RL == kAlongDepth) {
    const int i = wn * (16 * NB) + 8 * (li >> 2) + (li & 3);
    ra[0] = S::SLICE + 128 * i + 16 * (lg ^ chunk_swizzle<true>(i));
  } else {
    const int k = 8 * lg + (li >> 2);
#pragma unroll
    for (int b = 0; b < NB; ++b) ra[b] = S::SLICE + BT * E * k + 32 * ((wn * NB + b) ^ block_swizzle<BT>(k)) + 8 * (li & 3);
  }
  auto transposed = [&](int at) {
    // rows 4 apart have the same swizzle (f leaves bit 2 of k out)
    const s16x4 x = read_transposed((__attribute__((address_space(3))) s16x4*)(smem + at));
    const s16x4 y = read_transposed((__attribute__((address_space(3))) s16x4*)(smem + at + 4 * BT * E));
    i32x4 v;
    __builtin_memcpy(&v, &x, 8);
    __builtin_memcpy(reinterpret_cast<char*>(&v) + 8, &y, 8);
    return v;
  };
  auto read1 = [&](int kt, int half, i32x4 (&x)[FR], int g) {
    const int buf = (kt & 1) * 2 * S::SLICE;
    if (g < MB) {
      if constexpr (LL == kAlongDepth)
        x[g] = *reinterpret_cast<const i32x4*>(smem + buf + (la[0] ^ (64 * half)) + 2048 * g);
      else
        x[g] = transposed(buf + la[g] + 32 * BT * E * half);
    } else {
      if constexpr (RL == kAlongDepth)
        x[g] = *reinterpret_cast<const i32x4*>(smem + buf + (ra[0] ^ (64 * half)) + 4096 * ((g - MB) >> 1) + 512 * ((g - MB) & 1));
      else
        x[g] = transposed(buf + ra[g - MB] + 32 * BT * E * half);
    }
  };

  Acc acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = Acc{0, 0, 0, 0};
  i32x4 x0[FR], x1[FR];

  auto mma1 = [&](const i32x4 (&x)[FR], int u) {
    // block rows in order, the columns of every other one reversed: each step changes one operand
    const int mb = u / NB, nb = (mb & 1) ? NB - 1 - u % NB : u % NB;
    acc[mb][nb] = M::mma(x[MB + nb], x[mb], acc[mb][nb]);
  };
  constexpr int kMma = MB * NB;
  // first half of stage kt
  auto first_half = [&](int kt) {
    OZ2_WAIT_LGKMCNT(0);
    OZ2_SCHED_FENCE();
#pragma unroll
    for (int u = 0; u < kMma; ++u) {
      mma1(x0, u);
      if constexpr (kMma >= 2 * FR) {
        if (u % 2 == 0 && u / 2 < FR) read1(kt, 1, x1, u / 2);
      } else {
        if (u < FR) read1(kt, 1, x1, u);
      }
      OZ2_SCHED_FENCE();
    }
  };
  // second half: MORE: copies of stage kt + 2; NEXT: reads of stage kt + 1
  auto second_half = [&](int kt, auto more, auto next) {
#pragma unroll
    for (int u = 0; u < kMma; ++u) {
      mma1(x1, u);
      if constexpr (decltype(more)::value) {
        if (u < 2 * COPIES) copy1(kt + 2, u);
      }
      if constexpr (decltype(next)::value) {
        if constexpr (kMma >= 2 * FR) {
          if (u % 2 == 0 && u / 2 < FR) read1(kt + 1, 0, x0, u / 2);
        } else {
          if (u < FR) read1(kt + 1, 0, x0, u);
        }
      }
      OZ2_SCHED_FENCE();
    }
  };
  // every wave's copies of the next stage have landed, and every wave is done with this one
  auto middle = [&]() {
    OZ2_WAIT_LGKMCNT(0);
    OZ2_WAIT_VMCNT(0);
    OZ2_SCHED_FENCE();
    __builtin_amdgcn_s_barrier();
    OZ2_SCHED_FENCE();
  };

  if (nk > 0) {
    const bool partial = last_depth < kDepth;
#pragma unroll
    for (int j = 0; j < 2 * COPIES; ++j) copy1(0, j);
    if (nk > 1) {
#pragma unroll
      for (int j = 0; j < 2 * COPIES; ++j) copy1(1, j);
      OZ2_WAIT_VMCNT(2 * COPIES);
    } else {
      OZ2_WAIT_VMCNT(0);
    }
    OZ2_SCHED_FENCE();
    __builtin_amdgcn_s_barrier();
    if (nk == 1 && partial) {
      clear_tail();
      __syncthreads();
    }
    OZ2_SCHED_FENCE();
#pragma unroll
    for (int g = 0; g < FR; ++g) read1(0, 0, x0, g);
    OZ2_SCHED_FENCE();
    for (int kt = 0; kt < nk - 2; ++kt) {
      first_half(kt);
      middle();
      second_half(kt, std::true_type{}, std::true_type{});
    }
    if (nk > 1) {
      first_half(nk - 2);
      middle();
      if (partial) {
        clear_tail();
        __syncthreads();
      }
      second_half(nk - 2, std::false_type{}, std::true_type{});
    }
    first_half(nk - 1);
    OZ2_WAIT_LGKMCNT(0);
    OZ2_SCHED_FENCE();
    second_half(nk - 1, std::false_type{}, std::false_type{});
  }

  // acc[mb][nb][v]: output row m0 + 16 MB wm + 16 mb + lane % 16; column n0 + 16 NB wn +
  // 32 (nb / 2) + 8 (lane / 16) + 4 (nb % 2) + v, or, right operand along the index,
  // 16 nb + 4 (lane / 16) + v.
  const long mrow = m0 + wm * (16 * MB) + li;
  if constexpr (OUT == kOutPlain && RL == kAlongIndex) {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const long m = mrow + 16 * mb;
      if (m >= rows) continue;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int n = n0 + wn * (16 * NB) + 16 * nb + 4 * lg;
        if (n >= cols) continue;
        T t[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) t[v] = static_cast<T>(static_cast<float>(acc[mb][nb][v]));
        T* const y = static_cast<T*>(e.y) + m * e.ldy + n;
        if (n + 4 <= cols) {
          __builtin_memcpy(y, t, sizeof(t));
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (n + v < cols) y[v] = t[v];
        }
      }
    }
  } else {
    auto finish = [&](auto act, auto full) {
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const long m = mrow + 16 * mb;
        if (m >= rows) continue;
#pragma unroll
        for (int nb = 0; nb < NB; nb += 2) {
          const int n = n0 + wn * (16 * NB) + 16 * nb + 8 * lg;
          if (n >= cols) continue;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(acc[mb][nb + (i >> 2)][i & 3]);
          finish8<T, decltype(act)::value, decltype(full)::value>(v, e, m, n, cols);
        }
      }
    };
    if (cols % 8 == 0)
      with_activation(e.act, [&](auto act) { finish(act, std::true_type{}); });
    else
      with_activation(e.act, [&](auto act) { finish(act, std::false_type{}); });
  }
}

template <typename M, typename T, int BT, int LL, int RL, int OUT>
static hipError_t launch_tile(const Product& pr, hipStream_t st) {
  typedef typename M::elem E;
  const int tiles_m = (pr.rows + BT - 1) / BT, tiles_n = (pr.cols + BT - 1) / BT;
  const dim3 grid(static_cast<unsigned>(tiles_m) * static_cast<unsigned>(tiles_n));
  hipLaunchKernelGGL((product_tile_kernel<M, T, BT, LL, RL, OUT>), grid, dim3(64 * Tile<BT>::WAVES), 0, st, pr.rows,
                     pr.cols, pr.depth, static_cast<const E*>(pr.left), pr.left_ld, static_cast<const E*>(pr.right),
                     pr.right_ld, pr.epi, tiles_m, tiles_n);
  return hipGetLastError();
}

template <typename M, typename T, int LL, int RL, int OUT>
static hipError_t launch_tiles(const Product& pr, hipStream_t st) {
  const long big = static_cast<long>((pr.rows + 255) / 256) * ((pr.cols + 255) / 256);
  return big >= kBigTiles ? launch_tile<M, T, 256, LL, RL, OUT>(pr, st) : launch_tile<M, T, 128, LL, RL, OUT>(pr, st);
}

template <typename M, typename T>
static hipError_t launch_float(const Product& pr, hipStream_t st) {
  if (!pr.left_along_index && !pr.right_along_index) return launch_tiles<M, T, kAlongDepth, kAlongDepth, kOutEpilogue>(pr, st);
  if (!pr.left_along_index) return launch_tiles<M, T, kAlongDepth, kAlongIndex, kOutPlain>(pr, st);
  if (pr.right_along_index) return launch_tiles<M, T, kAlongIndex, kAlongIndex, kOutPlain>(pr, st);
  return hipErrorInvalidValue;
}

hipError_t launch_product(const Product& pr, hipStream_t st) {
  if (pr.i8) {
    if (pr.left_along_index || pr.right_along_index) return hipErrorInvalidValue;
    return pr.type == kTypeBf16 ? launch_tiles<MmaI8, bf16, kAlongDepth, kAlongDepth, kOutEpilogue>(pr, st)
                                : launch_tiles<MmaI8, f16, kAlongDepth, kAlongDepth, kOutEpilogue>(pr, st);
  }
  return pr.type == kTypeBf16 ? launch_float<MmaBf16, bf16>(pr, st) : launch_float<MmaF16, f16>(pr, st);
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
