// oz2_linear_tile.hpp -- out = epilogue(left right^T), the products of the linear layer and of
// its gradient: bf16 and f16 operands with f32 accumulators, int8 operands with int32 ones
// (exact: 127^2 times the depth stays below 2^31 up to the 2^17 the entry points accept).
// A header, so that each operand type is a translation unit of its own.
#pragma once

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

// What the tile kernel does with its accumulators: the whole epilogue; rounding and storing
// only; or storing them as they are, one of several sums over parts of the depth, which
// join_kernel adds up and finishes; or the third if there is a place for partial sums, else
// the second.
enum { kOutEpilogue = 0, kOutPlain = 1, kOutPartial = 2, kOutEither = 3 };

// How an operand lies in memory: along the depth (element (i, k) at i * ld + k), or along its
// own index (at k * ld + i), as W does in dX = dZ W and both operands do in dW = dZ^T X.
enum { kAlongDepth = 0, kAlongIndex = 1 };

// ---- tile kernel ---------------------------------------------------------------------
// BM x BN outputs per workgroup, its waves in a grid of WM x WN.  Depth advances in
// stages of 128 bytes, so that every row of an operand along the depth brings whole cache
// lines; a ring of two or four stages is held in LDS, filled with 1 KiB copies straight from memory.
//
// Per stage and wave, two halves of 64 bytes of depth (one matrix instruction deep):
//   first half:  MFMAs on the first fragments, the second half's fragments read between them;
//   middle:      every wave has read the stage: wait for the copies of the next stage, barrier;
//   second half: MFMAs on the second fragments, between them the copies of the stage one ring
//                ahead into the buffer just released, and the next stage's first fragments.
// So there is one barrier per stage, and a copy has the MFMAs of all but one stage of the ring
// to arrive.
//
// LDS layouts and bank conflicts.  Along the depth: rows of 128 bytes, 16-byte chunk c of row
// i at chunk c ^ s(i).  The 16 lanes that read one chunk of 16 rows then hit 16 different
// 16-byte bank groups (64 banks of 4 bytes): rows alternate between the halves of the banks
// by their lowest bit, and s takes 8 values over those with the same one.  The right operand's
// rows are dealt to the fragments so that a lane ends up with eight consecutive output
// columns (block b of a pair takes rows 8 g + 4 b + v of 32, g = 0..3, v = 0..3), and its s is
// chosen for that set.  Along the index: depth rows of BM (BN) elements, 32-byte block c of row
// k at block c ^ f(k), read with the transposing LDS read: 16 lanes fetch 4 depth rows x 16
// indices, each lane 8 bytes, and each receives one index's 4 depths.  f takes 16 values
// (256 elements), or 8 within either half of the wave (128 elements, 8 blocks), over the rows one
// read touches.
//
// With two groups of waves (GROUPS = 2), each takes one half of every stage for all of the tile
// and their sums meet in LDS at the end: one wave to a SIMD issues matrix instructions of this
// size at half rate only, two reach the full rate, and dividing the tile among eight waves
// instead would read LDS half as much again.
//
// What bounds it: the matrix cores, 70 to 74% busy at depth 8192 (LDS is active 27% of the time,
// without bank conflicts in the loop); at depth 2048 the epilogue's instructions and stores as well
// (58% busy in bf16, 43% in int8), which no other workgroup's products overlap.  Measured (bf16,
// on several boards): 8192^3 in 720 to 780 us, 1.41 to 1.53 PFLOP/s; 8192 x 2048 outputs at depth
// 8192 in 191 to 207 us in the three layouts, 1.33 to 1.44 PFLOP/s; int8 8192^3 in 380 to 438 us,
// 2.5 to 2.9 POP/s; 1024 x 4096 at depth 2048 (256 tiles of 128 x 128, one to a CU) in 21.3 to 21.8
// us, 0.8 PFLOP/s.  32 x 32 matrix
// instructions took 905 us for the first where these took 814, both before later steps.
constexpr int kStageBytes = 128;

template <int BM_, int BN_, int WM_, int WN_, int GROUPS_, int RING_, int PER_CU_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, GROUPS = GROUPS_;
  static constexpr int RING = RING_;            // stages in LDS
  static constexpr int PER_CU = PER_CU_;        // workgroups that fit a CU's LDS
  static constexpr int WAVES = WM * WN * GROUPS;
  static constexpr int MB = BM / (16 * WM);     // 16-row blocks per wave
  static constexpr int NB = BN / (16 * WN);     // 16-column blocks per wave
  static constexpr int LEFT = BM * kStageBytes;          // bytes of the left operand's stage, the right one's behind it
  static constexpr int STAGE = (BM + BN) * kStageBytes;
  static constexpr int LCOPIES = BM * kStageBytes / 1024 / WAVES, RCOPIES = BN * kStageBytes / 1024 / WAVES;  // 1 KiB copies per wave
  static_assert(BM * kStageBytes % (1024 * WAVES) == 0 && BN * kStageBytes % (1024 * WAVES) == 0 && NB % 2 == 0, "tile shape");
  static_assert(RING == 2 || RING == 4, "the waits assume these");
  static_assert(GROUPS == 1 || (MB % 2 == 0 && 8192 * (MB / 2) * NB <= RING * STAGE), "the groups' exchange");
};
// 128 x 64 outputs per wave, two waves to a SIMD: a stage is 2048 cycles of MFMAs, enough for the
// copies of the next to arrive.
typedef Tile<256, 256, 2, 4, 1, 2, 1> Tile256;
// Two workgroups to a CU, which have its matrix cores in turn: again 1024 cycles a stage each.
typedef Tile<128, 128, 2, 2, 1, 2, 2> Tile128;
// Alone on a CU: a stage is 512 cycles of MFMAs, so three more are under way.
typedef Tile<128, 128, 2, 2, 2, 4, 1> Tile128Deep;
typedef Tile<64, 128, 1, 4, 2, 4, 1> Tile64;

// s(i) of an operand along the depth.
template <bool RIGHT>
__device__ __forceinline__ int chunk_swizzle(int i) {
  return RIGHT ? (((i >> 3) & 3) << 1) | ((i >> 1) & 1) : (i >> 1) & 7;
}
// f(k) of an operand along the index, depth rows of B elements.
template <int B>
__device__ __forceinline__ int block_swizzle(int k) {
  static_assert(B == 128 || B == 256, "64-row tiles take their left operand along the depth");
  return B == 256 ? (k & 3) | (((k >> 3) & 3) << 2) : (k & 3) | (((k >> 3) & 1) << 2);
}

// Byte offset, from the operand's tile origin in a stage, of the 16 bytes that lane `lane`
// copies with the 1 KiB unit u.  Of a stage with `valid` elements of depth, chunks beyond them
// read something inside the operand (and are zeroed in LDS afterwards); so do rows beyond the
// last, and columns beyond the last chunk, which only reach outputs that are not stored.
template <int B, int E, int LAYOUT, bool RIGHT>
__device__ __forceinline__ unsigned copy_offset(int u, int lane, unsigned ld, int last_index, int valid) {
  if constexpr (LAYOUT == kAlongDepth) {
    const int i = 8 * u + (lane >> 3);
    const int c = (lane & 7) ^ chunk_swizzle<RIGHT>(i);
    return static_cast<unsigned>(min(i, last_index)) * ld * E + (c * (16 / E) < valid ? 16 * c : 0);
  } else {
    constexpr int kRow = B * E, kPerRow = kRow / 16;  // bytes and 16-byte chunks of a depth row
    const int k = u * (1024 / kRow) + lane / kPerRow;
    const int pc = lane % kPerRow;
    const int c = 2 * ((pc >> 1) ^ block_swizzle<B>(k)) + (pc & 1);
    return static_cast<unsigned>(min(k, valid - 1)) * ld * E + min(16 * c, last_index / (16 / E) * 16);
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

// The transposing read of 8 bytes per lane.  A function with a restrict pointer, so that the
// load carries aliasing information: without any, the compiler makes it wait for every copy
// into LDS that is still in flight.
__device__ __forceinline__ s16x4 read_transposed(__attribute__((address_space(3))) s16x4* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}

// One workgroup: tile number wg, stages kt0 .. kt0 + per - 1 of the depth (as many as there
// are), kt0 = per * part.  smem: RING stages.
template <typename M, typename T, typename S, int LL, int RL, int OUT, bool ADAPT = false>
__device__ __forceinline__ void product_tile(char* smem, unsigned wg, int part, int rows, int cols, int depth, int per,
                                             const typename M::elem* __restrict__ left, long left_ld,
                                             const typename M::elem* __restrict__ right, long right_ld,
                                             const Epilogue& e, typename M::acc* __restrict__ partial, int tiles_m,
                                             int tiles_n, const Adapters* ad = nullptr) {
  typedef typename M::acc Acc;
  constexpr int E = sizeof(typename M::elem);
  constexpr int kDepth = kStageBytes / E;  // elements of depth per stage
  constexpr int MB = S::MB, NB = S::NB, FR = MB + NB, LC = S::LCOPIES, COPIES = S::LCOPIES + S::RCOPIES;
  constexpr int kMask = S::RING - 1;  // stage kt lies in buffer kt & kMask
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // (256 x 256) waves w and w + 4 share a SIMD: the same rows, so the left fragments repeat there
  const int wm = wave % S::WM, wn = wave / S::WM % S::WN;
  const int group = S::GROUPS == 1 ? 0 : wave / (S::WM * S::WN);
  int ti, tj;
  tile_of(wg, tiles_m, tiles_n, ti, tj);
  const long m0 = static_cast<long>(ti) * S::BM;
  const int n0 = tj * S::BN;

  const int all = (depth + kDepth - 1) / kDepth, kt0 = per * part;
  const int nk = min(per, all - kt0);
  // elements of depth in this workgroup's last stage
  const int last_depth = kt0 + nk == all ? depth - (all - 1) * kDepth : kDepth;
  const long lstep = LL == kAlongDepth ? kStageBytes : kDepth * left_ld * E;
  const long rstep = RL == kAlongDepth ? kStageBytes : kDepth * right_ld * E;
  const char* const lbase = reinterpret_cast<const char*>(left) + (LL == kAlongDepth ? m0 * left_ld : m0) * E + kt0 * lstep;
  const char* const rbase = reinterpret_cast<const char*>(right) + (RL == kAlongDepth ? n0 * right_ld : n0) * E + kt0 * rstep;
  const int last_m = static_cast<int>(min(static_cast<long>(rows) - 1 - m0, static_cast<long>(S::BM - 1)));
  const int last_n = min(cols - 1 - n0, S::BN - 1);
  // read here: its use comes before that of y, whose load the output's pass through LDS hides
  float scale = 1.0f;
  if constexpr (OUT == kOutPlain || OUT == kOutEither) {
    scale = e.drop.scale;
    asm volatile("" : "+s"(scale));
  }
  unsigned off[COPIES];
  auto set_offsets = [&](int valid) {
#pragma unroll
    for (int j = 0; j < COPIES; ++j) {
      if (j < LC)
        off[j] = copy_offset<S::BM, E, LL, false>(wave + S::WAVES * j, lane, static_cast<unsigned>(left_ld), last_m, valid);
      else
        off[j] = copy_offset<S::BN, E, RL, true>(wave + S::WAVES * (j - LC), lane, static_cast<unsigned>(right_ld), last_n, valid);
    }
  };
  // copy j (the left operand's first) of stage kt into its buffer
  auto copy1 = [&](int kt, int j) {
    char* const dst = smem + (kt & kMask) * S::STAGE + (j < LC ? 0 : S::LEFT) + (wave + S::WAVES * (j < LC ? j : j - LC)) * 1024;
    const char* const src = j < LC ? lbase + kt * lstep : rbase + kt * rstep;
    // opaque, so that the address stays a scalar base and a 32-bit offset per lane (the compiler
    // otherwise keeps 64-bit lane pointers through the loop, and spills)
    unsigned o = off[j];
    asm volatile("" : "+v"(o));
    __builtin_amdgcn_global_load_lds(static_cast<const void*>(src + o), (lds_ptr_t)dst, 16, 0, 0);
  };
  // zeroes what lies beyond the depth in the last stage's buffer
  auto clear_tail = [&]() {
    constexpr int kChunks = kStageBytes / 16;
    char* const buf = smem + ((nk - 1) & kMask) * S::STAGE;
    for (int n = tid; n < S::STAGE / 16; n += 64 * S::WAVES) {
      const bool r = n >= S::LEFT / 16;
      const int c = r ? n - S::LEFT / 16 : n;
      bool beyond;
      if ((r ? RL : LL) == kAlongDepth)
        beyond = (c % kChunks ^ (r ? chunk_swizzle<true>(c / kChunks) : chunk_swizzle<false>(c / kChunks))) *
                     (16 / E) >= last_depth;
      else
        beyond = c / ((r ? S::BN : S::BM) * E / 16) >= last_depth;
      if (beyond) *reinterpret_cast<i32x4*>(buf + 16 * n) = i32x4{0, 0, 0, 0};
    }
  };

  // fragment reads
  const int li = lane & 15, lg = lane >> 4;
  // byte addresses of a lane's first block; the others are 16 rows (left) or 4 and 32 rows (right)
  // further along the depth, and along the index, where the block number only meets bits 5 to 8,
  // differ from it by exclusive or with 32 times theirs
  int la, ra;
  if constexpr (LL == kAlongDepth) {
    const int i = wm * (16 * MB) + li;
    la = kStageBytes * i + 16 * (lg ^ chunk_swizzle<false>(i));
  } else {
    const int k = 8 * lg + (li >> 2);
    la = S::BM * E * k + 32 * ((wm * MB) ^ block_swizzle<S::BM>(k)) + 8 * (li & 3);
  }
  if constexpr (RL == kAlongDepth) {
    const int i = wn * (16 * NB) + 8 * (li >> 2) + (li & 3);
    ra = S::LEFT + kStageBytes * i + 16 * (lg ^ chunk_swizzle<true>(i));
  } else {
    const int k = 8 * lg + (li >> 2);
    ra = S::LEFT + S::BN * E * k + 32 * ((wn * NB) ^ block_swizzle<S::BN>(k)) + 8 * (li & 3);
  }
  static_assert(S::LEFT % 512 == 0 && S::STAGE % 512 == 0 && (MB & (MB - 1)) == 0 && (NB & (NB - 1)) == 0, "block addresses");
  auto transposed = [&](int at, int row) {
    // rows 4 apart have the same swizzle (f leaves bit 2 of k out)
    const s16x4 x = read_transposed((__attribute__((address_space(3))) s16x4*)(smem + at));
    const s16x4 y = read_transposed((__attribute__((address_space(3))) s16x4*)(smem + at + 4 * row));
    i32x4 v;
    __builtin_memcpy(&v, &x, 8);
    __builtin_memcpy(reinterpret_cast<char*>(&v) + 8, &y, 8);
    return v;
  };
  auto read1 = [&](int kt, int half, i32x4 (&x)[FR], int g) {
    const int buf = (kt & kMask) * S::STAGE;
    if (g < MB) {
      if constexpr (LL == kAlongDepth)
        x[g] = *reinterpret_cast<const i32x4*>(smem + buf + (la ^ (64 * half)) + 16 * kStageBytes * g);
      else
        x[g] = transposed(((buf + la) ^ (32 * g)) + 32 * S::BM * E * half, S::BM * E);
    } else {
      if constexpr (RL == kAlongDepth)
        x[g] = *reinterpret_cast<const i32x4*>(smem + buf + (ra ^ (64 * half)) + 32 * kStageBytes * ((g - MB) >> 1) + 4 * kStageBytes * ((g - MB) & 1));
      else
        x[g] = transposed(((buf + ra) ^ (32 * (g - MB))) + 32 * S::BN * E * half, S::BN * E);
    }
  };

  Acc acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = Acc{0, 0, 0, 0};
  i32x4 x0[FR], x1[FR];

  // Adapters: the sums start from S_m B_a^T, worked out while the first stages' copies are under way.
  // A wave goes through the adapters of its rows, 64 at a time; where the depth has several parts or the
  // tile two groups of waves, these share the adapters.  Fragments come straight from memory (a cache,
  // mostly), and their products go to the rows that are the adapter's by selection, not by zeros in S:
  // an infinity in one request's adapter stays out of the others' rows.  S comes as two terms of the operands'
  // type (split_terms), each of which meets B.
  // Order matters: loads return in order, and the first stages' copies keep a tile's start busy.  The
  // rows' adapters and S (which no adapter's number is needed for) are asked for before the copies,
  // the first adapter's B behind the first stage's.
  // The rank goes by in steps of 32; a 64-row tile, whose rows are those of many requests, holds two (64
  // rows with adapters of their own, rank 64, 4096 -> 4096: 37.4 us for the call against 52.4 with one; 128- and
  // 256-row tiles spill).
  // Measured: 8192 x 8192 outputs at depth 2048, 24 requests, bias and gelu, with S's 12 to 20 us in it, 266 us at
  // rank 16, 278 at 32 and 317 at 64 (f16: 333), where the product alone takes 229: bound by what a tile waits for
  // before its first stage, four times.  37 rows with adapters of their own, rank 32, 8192 -> 2048, 11.4 us (10.0
  // without).
  constexpr bool kUnits = ADAPT && std::is_same_v<T, f16>;
  int own[ADAPT ? MB / 4 : 1];  // the adapter of row 64 h + lane of the wave's
  constexpr int kSteps = S::BM == 64 ? 2 : 1;  // of 32 elements of rank, held at a time
  i32x4 sf[kSteps][4][2];       // S of four blocks of rows, both terms
  float unit[4];
  i32x4 bf[kSteps][NB];         // B of `held`
  int held = -1, held_s = 0;    // S of 64 h + k0 / 32
  const int shares = static_cast<int>(gridDim.y) * S::GROUPS, share = part * S::GROUPS + group;
  constexpr bool kAlone = S::BM == 256;  // one part, one group of waves
  // (places beyond the rank are read inside it and set to zero; rows and columns outside the output are
  // computed, not stored)
  auto load_b = [&](int adapter, int k0) {
    const T* const b = static_cast<const T*>(ad->b) + adapter * ad->stride_b;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int col = min(n0 + wn * (16 * NB) + 32 * (nb >> 1) + 4 * (nb & 1) + 8 * (li >> 2) + (li & 3), cols - 1);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int k = k0 + 32 * i + 8 * lg;
        if (i == 0 || k0 + 32 * i < ad->rank) __builtin_memcpy(&bf[i][nb], b + col * ad->ldb + (k < ad->rank ? k : 0), 16);
      }
    }
    held = adapter;
  };
  const int pitch = ADAPT ? ad->pitch() : 0;
  const char* const s_base = ADAPT ? static_cast<const char*>(ad->s) + 4 * m0 * pitch : nullptr;
  auto load_s = [&](int h, int k0) {
#pragma unroll
    for (int mb = 0; mb < 4; ++mb) {
      const int m = min(wm * (16 * MB) + 64 * h + 16 * mb + li, last_m);  // of the tile's rows
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int k = k0 + 32 * i + 8 * lg;
        if (i > 0 && k0 + 32 * i >= ad->rank) continue;
        const unsigned at = 4u * (m * pitch + (k < pitch ? k : 0));
#pragma unroll
        for (int term = 0; term < 2; ++term) sf[i][mb][term] = *reinterpret_cast<const i32x4*>(s_base + at + 16 * term);
      }
      if constexpr (kUnits) unit[mb] = ad->unit[(m0 + m) * ad->blocks() + k0 / 64];
    }
    held_s = 64 * h + k0 / 32;
  };
  // rows of group h whose adapter is this part's and group of waves's to add
  auto shared_rows = [&](int h) {
    return __ballot(own[h] >= 0 && own[h] < ad->count && (kAlone || own[h] % shares == share));
  };
  auto adapters_early = [&]() {
#pragma unroll
    for (int h = 0; h < MB / 4; ++h) {
      const long m = m0 + wm * (16 * MB) + 64 * h + lane;
      own[h] = m < rows ? ad->index[m] : -1;
    }
    load_s(0, 0);
  };
  auto adapters_first = [&]() {
    const unsigned long todo = shared_rows(0);
    if (todo != 0) load_b(__builtin_amdgcn_readlane(own[0], __builtin_ctzl(todo)), 0);
  };
  auto adapters_term = [&]() {
    static_assert(!ADAPT || (E == 2 && LL == kAlongDepth && RL == kAlongDepth && MB % 4 == 0), "16-bit operands along the depth");
    const int rank = ad->rank;
#pragma unroll
    for (int h = 0; h < MB / 4; ++h) {
      for (unsigned long todo = shared_rows(h); todo != 0;) {
        const int adapter = __builtin_amdgcn_readlane(own[h], __builtin_ctzl(todo));
        const unsigned long match = __ballot(own[h] == adapter);
        todo &= ~match;
        for (int k0 = 0; k0 < rank; k0 += 32 * kSteps) {
          if (h > 0 || k0 > 0 || held != adapter) load_b(adapter, k0);  // (kept over the groups of rows it is spilled)
          if (held_s != 64 * h + k0 / 32) load_s(h, k0);
          OZ2_SCHED_FENCE();
          const i32x4 zero = {0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) bf[i][nb] = k0 + 32 * i + 8 * lg < rank ? bf[i][nb] : zero;
#pragma unroll
          for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
              for (int term = 0; term < 2; ++term) sf[i][mb][term] = k0 + 32 * i + 8 * lg < pitch ? sf[i][mb][term] : zero;
            const bool mine = match >> (16 * mb + li) & 1;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              Acc& a = acc[4 * h + mb][nb];
              Acc t = kUnits ? Acc{0, 0, 0, 0} : a;
#pragma unroll
              for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int term = 0; term < 2; ++term)
                  if (i == 0 || k0 + 32 * i < rank) t = M::mma(bf[i][nb], sf[i][mb][term], t);
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                float sum = t[v];
                if constexpr (kUnits) sum = __builtin_fmaf(t[v], unit[mb], a[v]);
                a[v] = mine ? sum : a[v];
              }
            }
            OZ2_SCHED_FENCE();
          }
        }
      }
    }
  };
  auto mma1 = [&](const i32x4 (&x)[FR], int u) {
    // block rows in order, the columns of every other one reversed: each step changes one operand
    const int mb = u / NB, nb = (mb & 1) ? NB - 1 - u % NB : u % NB;
    acc[mb][nb] = M::mma(x[MB + nb], x[mb], acc[mb][nb]);
  };
  constexpr int kMma = MB * NB;
  // fragment reads after every second MFMA where there are enough of them, else spread evenly
  auto reads = [&](int kt, int half, i32x4 (&x)[FR], int u) {
    if constexpr (kMma >= 2 * FR) {
      if (u % 2 == 0 && u / 2 < FR) read1(kt, half, x, u / 2);
    } else {
#pragma unroll
      for (int g = u * FR / kMma; g < (u + 1) * FR / kMma; ++g) read1(kt, half, x, g);
    }
  };
  // copies of stage kt + RING, spread over a half's MFMAs: issued together at its start they hold
  // up every wave's MFMAs behind 64 KiB of copies (8192 x 8192 outputs at depth 2048: 212 us
  // against 228; 8192 x 2048 at depth 8192, right operand along the index, 202 against 219)
  constexpr int kEvery = kMma / COPIES;
  static_assert(kMma >= COPIES, "a copy per MFMA at most");
  auto copies = [&](int kt, bool more, int u) {
    if (u % kEvery == 0 && u / kEvery < COPIES) {
      if (more) copy1(kt + S::RING, u / kEvery);
    }
  };
  // first half of stage kt
  auto first_half = [&](int kt) {
    OZ2_WAIT_LGKMCNT(0);
    OZ2_SCHED_FENCE();
#pragma unroll
    for (int u = 0; u < kMma; ++u) {
      mma1(x0, u);
      reads(kt, 1, x1, u);
      OZ2_SCHED_FENCE();
    }
  };
  // second half: copies of stage kt + RING (if there is one), reads of stage kt + 1 (past the last
  // stage, of a buffer whose contents are not used)
  auto second_half = [&](int kt) {
    const bool more = kt + S::RING < nk;
#pragma unroll
    for (int u = 0; u < kMma; ++u) {
      mma1(x1, u);
      copies(kt, more, u);
      reads(kt + 1, 0, x0, u);
      OZ2_SCHED_FENCE();
    }
  };
  // this wave's copies of stage `ready` have landed: of the later ones, those under way (no
  // more than RING - 1 stages beyond it, of nk in all) may still be
  auto wait_copies = [&](int ready, int under_way) {
    const int later = min(under_way, nk - 1 - ready);
    if (later <= 0)
      OZ2_WAIT_VMCNT(0);
    else if (later == 1)
      OZ2_WAIT_VMCNT(COPIES);
    else if (later == 2)
      OZ2_WAIT_VMCNT(2 * COPIES);
    else
      OZ2_WAIT_VMCNT(3 * COPIES);
  };
  // every wave's copies of the next stage have landed, and every wave is done with this one
  auto middle = [&](int kt) {
    OZ2_WAIT_LGKMCNT(0);
    if constexpr (S::RING == 2)
      OZ2_WAIT_VMCNT(0);
    else
      wait_copies(kt + 1, S::RING - 2);
    OZ2_SCHED_FENCE();
    __builtin_amdgcn_s_barrier();
    OZ2_SCHED_FENCE();
  };

  if (nk > 0) {
    const bool partial = last_depth < kDepth;
    set_offsets(kDepth);
    if constexpr (ADAPT) adapters_early();
#pragma unroll
    for (int kt = 0; kt < S::RING; ++kt) {
      if (kt >= nk) break;
      if (kt == nk - 1) set_offsets(last_depth);
#pragma unroll
      for (int j = 0; j < COPIES; ++j) copy1(kt, j);
      if constexpr (ADAPT) {
        if (kt == 0) adapters_first();
      }
    }
    if constexpr (ADAPT) {
      // The condition holds whenever this kernel runs.  It is called unlikely so that the compiler, which
      // takes nested loops for the hot part, does not spill in the loop over the depth, where a reload
      // waits for the copies under way, or between the epilogue's stores, where it waits for them (490 us and
      // more for 8192 x 8192 outputs).
      if (__builtin_expect_with_probability(ad->rank > 0, 0, 1.0)) adapters_term();
    }
    wait_copies(0, S::RING - 1);
    OZ2_SCHED_FENCE();
    __builtin_amdgcn_s_barrier();
    if (nk == 1 && partial) {
      clear_tail();
      __syncthreads();
    }
    OZ2_SCHED_FENCE();
    if constexpr (S::GROUPS == 1) {
#pragma unroll
      for (int g = 0; g < FR; ++g) read1(0, 0, x0, g);
      OZ2_SCHED_FENCE();
      // one loop body for every stage: peeled ends cost the compiler a second set of registers
      for (int kt = 0; kt < nk; ++kt) {
        // opaque, so that the blocks' addresses are worked out at each read and not all kept in
        // registers (which spill, and a reload waits for the copies under way)
        if constexpr (LL == kAlongIndex) asm volatile("" : "+v"(la));
        if constexpr (RL == kAlongIndex) asm volatile("" : "+v"(ra));
        first_half(kt);
        if (kt == nk - 1 - S::RING) set_offsets(last_depth);
        middle(kt);
        if (kt == nk - 2 && partial) {
          clear_tail();
          __syncthreads();
        }
        second_half(kt);
      }
    } else {
#pragma unroll
      for (int g = 0; g < FR; ++g) read1(0, group, x0, g);
      OZ2_SCHED_FENCE();
      // this group's half of a stage: fragments x, reading the next stage's into y
      auto stage = [&](int kt, const i32x4 (&x)[FR], i32x4 (&y)[FR]) {
        if (kt == nk - 1 - S::RING) set_offsets(last_depth);
        middle(kt);
        if (kt == nk - 2 && partial) {
          clear_tail();
          __syncthreads();
        }
        const bool more = kt + S::RING < nk;
#pragma unroll
        for (int u = 0; u < kMma; ++u) {
          mma1(x, u);
          copies(kt, more, u);
          reads(kt + 1, group, y, u);
          OZ2_SCHED_FENCE();
        }
      };
      for (int kt = 0; kt < nk; kt += 2) {
        stage(kt, x0, x1);
        if (kt + 1 < nk) stage(kt + 1, x1, x0);
      }
    }
    OZ2_WAIT_LGKMCNT(0);
  }
  // Two groups: each gives the other half of its blocks and finishes the other half.
  constexpr int EMB = S::GROUPS == 1 ? MB : MB / 2;
  Acc sum[EMB][NB];
  if constexpr (S::GROUPS == 1) {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) sum[mb][nb] = acc[mb][nb];
  } else {
    Acc* const slots = reinterpret_cast<Acc*>(smem);
    __syncthreads();
#pragma unroll
    for (int mb = 0; mb < EMB; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        slots[((wave ^ (S::WAVES / 2)) * EMB * NB + mb * NB + nb) * 64 + lane] = group == 0 ? acc[mb + EMB][nb] : acc[mb][nb];
    __syncthreads();
#pragma unroll
    for (int mb = 0; mb < EMB; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        sum[mb][nb] = (group == 0 ? acc[mb][nb] : acc[mb + EMB][nb]) + slots[(wave * EMB * NB + mb * NB + nb) * 64 + lane];
  }

  // sum[mb][nb][v]: output row m0 + 16 MB wm + 16 EMB group + 16 mb + lane % 16; column n0 + 16 NB wn +
  // 32 (nb / 2) + 8 (lane / 16) + 4 (nb % 2) + v, or, right operand along the index,
  // 16 nb + 4 (lane / 16) + v.
  // The lane's place is worked out again here rather than kept in registers through the loop.
  int end_tid = threadIdx.x;
  asm volatile("" : "+v"(end_tid));
  const int end_lane = end_tid & 63;
  const int eg = end_lane >> 4;
  const long mrow = m0 + wm * (16 * MB) + group * (16 * EMB) + (end_lane & 15);
  if (OUT == kOutPartial || (OUT == kOutEither && partial != nullptr)) {
    // the sums as they are, rows of cols rounded up to a multiple of 8
    const long ld4 = (cols + 7) / 8 * 2;
    Acc* const dst = partial + part * (rows * ld4);
#pragma unroll
    for (int mb = 0; mb < EMB; ++mb) {
      const long m = mrow + 16 * mb;
      if (m >= rows) continue;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int n = n0 + wn * (16 * NB) + (RL == kAlongDepth ? 32 * (nb >> 1) + 8 * eg + 4 * (nb & 1) : 16 * nb + 4 * eg);
        if (n < cols) dst[m * ld4 + n / 4] = sum[mb][nb];
      }
    }
    return;
  }
  if constexpr (OUT == kOutPlain || OUT == kOutEither) {
    static_assert(RL == kAlongIndex, "the column order below");
    // Through LDS, so that a store instruction writes whole rows of the tile: a lane's own four
    // columns are 8 bytes, and stored directly they cost as much again as a launch (1024 x 256
    // outputs at depth 64: 9.0 us against 5.6 without stores).  16-byte chunk c of row i lies
    // at chunk c ^ (i mod 16).
    constexpr int kChunks = S::BN / 8, kPitch = 2 * S::BN;
    static_assert(S::BM * kPitch <= S::RING * S::STAGE, "the tile fits the ring");
    __syncthreads();
#pragma unroll
    for (int mb = 0; mb < EMB; ++mb) {
      const int i = static_cast<int>(mrow - m0) + 16 * mb;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int c = wn * (2 * NB) + 2 * nb + (eg >> 1);
        T t[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) t[v] = static_cast<T>(scale * static_cast<float>(sum[mb][nb][v]));
        __builtin_memcpy(smem + i * kPitch + 16 * (c ^ (i & 15)) + 8 * (eg & 1), t, sizeof(t));
      }
    }
    __syncthreads();
    const int c = end_tid % kChunks, n = n0 + 8 * c;
    if (n >= cols) return;
#pragma unroll
    for (int i = end_tid / kChunks; i < S::BM; i += 64 * S::WAVES / kChunks) {
      if (m0 + i >= rows) break;
      raw8 r;
      __builtin_memcpy(&r, smem + i * kPitch + 16 * (c ^ (i & 15)), 16);
      T* const y = static_cast<T*>(e.y) + (m0 + i) * e.ldy + n;
      if (n + 8 <= cols) {
        store16<false>(y, r);
      } else {
        T t[8];
        __builtin_memcpy(t, &r, 16);
#pragma unroll
        for (int v = 0; v < 8; ++v)
          if (n + v < cols) y[v] = t[v];
      }
    }
  } else if constexpr (OUT == kOutEpilogue) {
    // Everything the epilogue reads is read first, for all of the wave's groups of eight columns:
    // the stores may alias it as far as the compiler knows (Y may be R), so it would wait for
    // each group's loads in turn.
    auto finish = [&](auto act, auto full) {
      constexpr bool FULL = decltype(full)::value;
      // 256 x 256 tiles run on large outputs only, which stream past the operands in the caches:
      // 243 us against 254 for 8192 x 8192 outputs at depth 2048 with gelu and Z
      constexpr bool NT = S::BM == 256;
      constexpr int NG = NB / 2;
      const int nfirst = n0 + wn * (16 * NB) + 8 * eg;
      raw8 bias[NG] = {}, res[EMB][NG] = {};
      float xs[EMB] = {}, ws[NG][8] = {};
      if (e.res != nullptr) {
#pragma unroll
        for (int mb = 0; mb < EMB; ++mb)
#pragma unroll
          for (int g = 0; g < NG; ++g)
            if (mrow + 16 * mb < rows && nfirst + 32 * g < cols)
              res[mb][g] = load_raw8<T, FULL>(e.res, (mrow + 16 * mb) * e.ldr + nfirst + 32 * g, cols - nfirst - 32 * g);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int n = nfirst + 32 * g;
        if (n >= cols) continue;
        if (e.bias != nullptr) bias[g] = load_raw8<T, FULL>(e.bias, n, cols - n);
        if constexpr (E == 1) load8(e.ws + n, FULL ? 8 : cols - n, ws[g]);
      }
      if constexpr (E == 1) {
#pragma unroll
        for (int mb = 0; mb < EMB; ++mb)
          if (mrow + 16 * mb < rows) xs[mb] = e.xs[mrow + 16 * mb];
      }
#pragma unroll
      for (int mb = 0; mb < EMB; ++mb) {
        const long m = mrow + 16 * mb;
        if (m >= rows) continue;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int n = nfirst + 32 * g;
          if (n >= cols) continue;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(sum[mb][2 * g + (i >> 2)][i & 3]);
          finish8<T, decltype(act)::value, FULL, NT>(v, e, m, n, cols, xs[mb], ws[g], bias[g], res[mb][g]);
        }
      }
    };
    if (cols % 8 == 0)
      with_activation(e.act, [&](auto act) { finish(act, std::true_type{}); });
    else
      with_activation(e.act, [&](auto act) { finish(act, std::false_type{}); });
  }
}

template <typename M, typename T, typename S, int LL, int RL, int OUT>
__global__ __launch_bounds__(64 * S::WAVES, S::PER_CU) void product_tile_kernel(
    int rows, int cols, int depth, int per, const typename M::elem* __restrict__ left, long left_ld,
    const typename M::elem* __restrict__ right, long right_ld, Epilogue e, typename M::acc* __restrict__ partial,
    int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) char smem[S::RING * S::STAGE];
  product_tile<M, T, S, LL, RL, OUT>(smem, blockIdx.x, blockIdx.y, rows, cols, depth, per, left, left_ld, right,
                                     right_ld, e, partial, tiles_m, tiles_n);
}

template <typename M, typename T, typename S, int OUT>
__global__ __launch_bounds__(64 * S::WAVES, S::PER_CU) void product_adapters_kernel(
    int rows, int cols, int depth, int per, const typename M::elem* __restrict__ left, long left_ld,
    const typename M::elem* __restrict__ right, long right_ld, Epilogue e, typename M::acc* __restrict__ partial,
    int tiles_m, int tiles_n, Adapters ad) {
  __shared__ __attribute__((aligned(1024))) char smem[S::RING * S::STAGE];
  product_tile<M, T, S, kAlongDepth, kAlongDepth, OUT, true>(smem, blockIdx.x, blockIdx.y, rows, cols, depth, per, left,
                                                             left_ld, right, right_ld, e, partial, tiles_m, tiles_n, &ad);
}

// Two gradient products and the column sums in one launch: dX = dZ W on the first workgroups,
// dW = dZ^T X on the next, the sums on the last, so that products of too few tiles to fill the
// CUs fill them together: 23.3 us for 1537 x 1001 and 2049 x 1001 outputs (240 tiles) with the
// sums, where the products alone, one after the other, took 21.4 and 18.5 (1000 columns).
template <typename M>
struct PairSide {
  int rows, cols, depth, per, tiles_m, tiles_n, parts;
  const typename M::elem* left;
  long left_ld;
  const typename M::elem* right;
  long right_ld;
  Epilogue epi;
  typename M::acc* partial;  // null: outputs are stored directly
  unsigned workgroups() const { return static_cast<unsigned>(tiles_m) * tiles_n * parts; }
};

template <typename M, typename T, typename S>
__global__ __launch_bounds__(64 * S::WAVES, S::PER_CU) void product_pair_kernel(PairSide<M> dx, PairSide<M> dw, ColumnSums sums) {
  __shared__ __attribute__((aligned(1024))) char smem[S::RING * S::STAGE];
  unsigned wg = blockIdx.x;
  const unsigned nx = static_cast<unsigned>(dx.tiles_m) * dx.tiles_n, nw = static_cast<unsigned>(dw.tiles_m) * dw.tiles_n;
  if (wg < nx * dx.parts) {
    product_tile<M, T, S, kAlongDepth, kAlongIndex, kOutEither>(smem, wg % nx, wg / nx, dx.rows, dx.cols, dx.depth, dx.per,
                                                                dx.left, dx.left_ld, dx.right, dx.right_ld, dx.epi,
                                                                dx.partial, dx.tiles_m, dx.tiles_n);
    return;
  }
  wg -= nx * dx.parts;
  if (wg < nw * dw.parts) {
    product_tile<M, T, S, kAlongIndex, kAlongIndex, kOutEither>(smem, wg % nw, wg / nw, dw.rows, dw.cols, dw.depth, dw.per,
                                                                dw.left, dw.left_ld, dw.right, dw.right_ld, dw.epi,
                                                                dw.partial, dw.tiles_m, dw.tiles_n);
    return;
  }
  wg -= nw * dw.parts;
  column_sums<T, 64 * S::WAVES>(reinterpret_cast<float*>(smem), wg, sums);
}

// Adds up the sums over parts of the depth, in their order, and finishes the outputs: eight
// columns of one row per thread.  Workgroups of one wave: there are few outputs, and a wave
// waits mostly for its loads (3.9 us for 37 x 2048 outputs in 16 parts, 4.8 MB).
constexpr int kJoinThreads = 64;

template <typename M, typename T, int ACT, bool FULL>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(int rows, int cols, int splits,
                                                            const typename M::acc* __restrict__ partial, Epilogue e) {
  const int groups = (cols + 7) / 8;
  const long plane = static_cast<long>(rows) * groups * 2;
  const long n = static_cast<long>(blockIdx.x) * kJoinThreads + threadIdx.x;
  if (n >= static_cast<long>(rows) * groups) return;
  const long m = n / groups;
  const int col = 8 * static_cast<int>(n - m * groups), valid = cols - col;
  // what the epilogue reads is under way with the sums
  float xs = 0.0f, ws[8] = {};
  raw8 bias = {}, res = {};
  if (e.res != nullptr) res = load_raw8<T, FULL>(e.res, m * e.ldr + col, valid);
  if (e.bias != nullptr) bias = load_raw8<T, FULL>(e.bias, col, valid);
  if constexpr (sizeof(typename M::elem) == 1) {
    xs = e.xs[m];
    load8(e.ws + col, FULL ? 8 : valid, ws);
  }
  typename M::acc a = partial[2 * n], b = partial[2 * n + 1];
#pragma unroll 8
  for (int s = 1; s < splits; ++s) {
    a += partial[s * plane + 2 * n];
    b += partial[s * plane + 2 * n + 1];
  }
  const float scale = e.drop.t == 0 ? e.drop.scale : 1.0f;
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = scale * static_cast<float>(a[i]);
    v[4 + i] = scale * static_cast<float>(b[i]);
  }
  finish8<T, ACT, FULL>(v, e, m, col, cols, xs, ws, bias, res);
}

template <typename M, typename T, typename S, int LL, int RL, int OUT>
static hipError_t launch_tile(const Product& pr, hipStream_t st) {
  typedef typename M::elem E;
  const int tiles_m = (pr.rows + S::BM - 1) / S::BM, tiles_n = (pr.cols + S::BN - 1) / S::BN;
  const int stages = (pr.depth * static_cast<int>(sizeof(E)) + kStageBytes - 1) / kStageBytes;
  const int per = OUT == kOutPartial ? (stages + pr.plan.splits - 1) / pr.plan.splits : stages;
  const dim3 grid(static_cast<unsigned>(tiles_m) * static_cast<unsigned>(tiles_n), OUT == kOutPartial ? pr.plan.splits : 1);
  hipLaunchKernelGGL((product_tile_kernel<M, T, S, LL, RL, OUT>), grid, dim3(64 * S::WAVES), 0, st, pr.rows, pr.cols,
                     pr.depth, per, static_cast<const E*>(pr.left), pr.left_ld, static_cast<const E*>(pr.right),
                     pr.right_ld, pr.epi, static_cast<typename M::acc*>(pr.partial), tiles_m, tiles_n);
  return hipGetLastError();
}

template <typename M, typename T>
static hipError_t launch_join(const Product& pr, hipStream_t st) {
  const long n = static_cast<long>(pr.rows) * ((pr.cols + 7) / 8);
  const dim3 grid(static_cast<unsigned>((n + kJoinThreads - 1) / kJoinThreads));
  with_activation(pr.epi.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    const auto kernel = pr.cols % 8 == 0 ? join_kernel<M, T, ACT, true> : join_kernel<M, T, ACT, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(kJoinThreads), 0, st, pr.rows, pr.cols, pr.plan.splits,
                       static_cast<const typename M::acc*>(pr.partial), pr.epi);
  });
  return hipGetLastError();
}

template <typename M>
static PairSide<M> pair_side(const Product& pr) {
  typedef Tile128Deep S;
  const int stages = (pr.depth * static_cast<int>(sizeof(typename M::elem)) + kStageBytes - 1) / kStageBytes;
  PairSide<M> side;
  side.rows = pr.rows;
  side.cols = pr.cols;
  side.depth = pr.depth;
  side.parts = pr.plan.splits;
  side.per = (stages + side.parts - 1) / side.parts;
  side.tiles_m = (pr.rows + S::BM - 1) / S::BM;
  side.tiles_n = (pr.cols + S::BN - 1) / S::BN;
  side.left = static_cast<const typename M::elem*>(pr.left);
  side.left_ld = pr.left_ld;
  side.right = static_cast<const typename M::elem*>(pr.right);
  side.right_ld = pr.right_ld;
  side.epi = pr.epi;
  side.partial = pr.plan.splits > 1 ? static_cast<typename M::acc*>(pr.partial) : nullptr;
  return side;
}

template <typename M, typename T>
static hipError_t launch_pair(const Product& dx, const Product& dw, const ColumnSums& sums, hipStream_t st) {
  typedef Tile128Deep S;
  const PairSide<M> px = pair_side<M>(dx), pw = pair_side<M>(dw);
  const unsigned n = px.workgroups() + pw.workgroups() + (sums.db != nullptr ? (sums.r + kSumColumns - 1) / kSumColumns : 0);
  hipLaunchKernelGGL((product_pair_kernel<M, T, S>), dim3(n), dim3(64 * S::WAVES), 0, st, px, pw, sums);
  hipError_t err = hipGetLastError();
  if (err == hipSuccess && dx.plan.splits > 1) err = launch_join<M, T>(dx, st);
  if (err == hipSuccess && dw.plan.splits > 1) err = launch_join<M, T>(dw, st);
  return err;
}

// One layout of the operands on the planned tile; OUT: kOutEpilogue or kOutPlain.
template <typename M, typename T, typename S, int LL, int RL, int OUT>
static hipError_t launch_split(const Product& pr, hipStream_t st) {
  if (pr.plan.splits <= 1) return launch_tile<M, T, S, LL, RL, OUT>(pr, st);
  const hipError_t err = launch_tile<M, T, S, LL, RL, kOutPartial>(pr, st);
  return err != hipSuccess ? err : launch_join<M, T>(pr, st);
}

template <typename M, typename T, int LL, int RL, int OUT>
static hipError_t launch_layout(const Product& pr, hipStream_t st) {
  switch (pr.plan.tile) {
    case kTile256:
      return launch_tile<M, T, Tile256, LL, RL, OUT>(pr, st);
    case kTile128:
      return launch_split<M, T, Tile128, LL, RL, OUT>(pr, st);
    case kTile128Deep:
      return launch_split<M, T, Tile128Deep, LL, RL, OUT>(pr, st);
    case kTile64:
      if constexpr (LL == kAlongDepth) return launch_split<M, T, Tile64, LL, RL, OUT>(pr, st);
      break;
  }
  return hipErrorInvalidValue;
}

// ---- few rows ----------------------------------------------------------------------------
// rows <= R, both operands along the depth, rows at any alignment.  Reading the right
// operand (the weights) once is the whole work, so it goes straight from memory to registers:
// a workgroup takes R of its rows and its waves share the depth, each with a contiguous part
// in steps, kDeep steps' loads in flight.  The waves' sums meet in LDS.  Bound by memory: one
// row on 8192 x 2048 bf16 weights 8.1 us, 4.1 TB/s with the launch in it; on 8192 x 8192, 24.4 us,
// 5.5 TB/s (a large copy moves 5.2 TB/s both ways).
// R = 16: a step is 64 bytes per row, one matrix instruction deep.  R = 8: the instruction's
// 16 rows and columns hold 8 rows twice, 64 bytes further along the second time, on both
// sides; the two diagonal quarters of its result are then sums over two parts of the depth
// (the others are not used).  That gives twice the workgroups, and whole cache lines per row.
// The matrix cores compute R rows whatever there are: at one instruction per KiB of weights
// they are far from busy.
// QUANT (int8): the left operand is still in the outputs' type; every workgroup quantises the
// few rows itself, into LDS, which saves a launch and hides behind the first loads of weights.
template <typename E>
__device__ __forceinline__ i32x4 load_chunk(const E* row, int k, int depth) {
  constexpr int N = 16 / sizeof(E);
  i32x4 v;
  if (k + N <= depth) {
    __builtin_memcpy(&v, row + k, 16);
  } else {
    E t[N];
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = k + i < depth ? row[k + i] : static_cast<E>(0);
    __builtin_memcpy(&v, t, 16);
  }
  return v;
}

constexpr int kFewWaves = 8;

// Element i of S, `count` elements to a part, the parts' loads four at a time (of a row without an
// adapter something that is not used).
__device__ __forceinline__ float adapter_sum(const Adapters& ad, int count, int i) {
  const float* const s = static_cast<const float*>(ad.s) + i;
  float sum = 0.0f;
  for (int j = 0; j < ad.parts; j += 4) {
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = s[static_cast<long>(min(j + u, ad.parts - 1)) * count];
#pragma unroll
    for (int u = 0; u < 4; ++u) sum += j + u < ad.parts ? v[u] : 0.0f;
  }
  return sum;
}

// ADAPT: the adapters' term, S and B read behind the first loads of weights: a thread per output adds
// up its row of B with its token's S, which goes through LDS.  One row on 8192 x 2048 weights, rank 16, takes as
// long as without (9.1 to 9.7 us in a trace).  B beyond the first 16 of rank is read behind the barrier, 8 elements at
// a time, and every workgroup adds up S's parts for itself: on 4096 x 8192 weights, S before it included, one row
// takes 17.4 us at rank 16, 18.4 at 32, 19.7 at 64 and 32 at 256 (12.9 without adapters); eight rows 20, 21, 23 and
// 41 (15.2); sixteen 26, 28, 30 and 47 (16.5).
template <typename M, typename T, int R, bool QUANT, int ACT, bool FULL, bool ADAPT = false>
__device__ __forceinline__ void product_few(int rows, int cols, int depth, int per, const void* __restrict__ left, long left_ld,
                                            const typename M::elem* __restrict__ right, long right_ld, Epilogue e,
                                            const Adapters* ad = nullptr) {
  typedef typename M::elem E;
  typedef typename M::acc Acc;
  constexpr int G = 16 / R, kStep = G * 64 / sizeof(E), kDeep = 8;
  __shared__ Acc sums[kFewWaves][16][4];  // wave, column, four rows each of the instruction's result
  __shared__ float out[R][R];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * R;
  const int li = lane & 15;
  const int k0 = (li / R) * (64 / static_cast<int>(sizeof(E))) + (lane >> 4) * (16 / static_cast<int>(sizeof(E)));
  const E* const rrow = right + min(n0 + li % R, cols - 1) * right_ld;
  const int lm = min(li % R, rows - 1);
  // adapters: thread m R + n has the output of row m, column n0 + n
  const T* brow = nullptr;
  if constexpr (ADAPT) {
    const int m = threadIdx.x / R, n = n0 + static_cast<int>(threadIdx.x) % R;
    const int a = m < rows && n < cols ? ad->index[m] : -1;
    if (a >= 0 && a < ad->count) brow = static_cast<const T*>(ad->b) + a * ad->stride_b + n * ad->ldb;
  }
  // this wave's steps: `per` of them, the last wave's the rest; whole steps in groups of kDeep
  const int steps = (depth + kStep - 1) / kStep, whole = depth / kStep;
  const int s0 = wave * per, s1 = min((wave + 1) * per, steps), s1w = min(s1, whole);
  i32x4 w[kDeep];
  auto load_weights = [&](int s) {
#pragma unroll
    for (int j = 0; j < kDeep; ++j) __builtin_memcpy(&w[j], rrow + (s + j) * kStep + k0, 16);
  };
  const bool deep = s0 + kDeep <= s1w;
  if (deep) load_weights(s0);

  // the first of B's row and of S are under way with the weights
  constexpr int kHeldRank = 16;
  raw8 held_b[kHeldRank / 8];
  float held_s = 0.0f;
  if constexpr (ADAPT) {
#pragma unroll
    for (int c = 0; c < kHeldRank / 8; ++c)
      if (brow != nullptr && 8 * c < ad->rank) held_b[c] = load_raw8<T, false>(brow, 8 * c, ad->rank - 8 * c);
    const int count = rows * ad->pitch();
    if (static_cast<int>(threadIdx.x) < count) held_s = adapter_sum(*ad, count, threadIdx.x);
  }

  extern __shared__ __attribute__((aligned(16))) int8_t levels[];  // QUANT: rows of `pitch` bytes; ADAPT: S
  const int pitch = (depth + 15) / 16 * 16;
  if constexpr (QUANT) {
    // the thread's first kHeld groups of eight of each row stay in registers where there is one row
    constexpr int kHeld = 2;
    __shared__ float tops[R][kFewWaves], scales[R];
    float held[kHeld][8], v[8];
    for (int m = 0; m < rows; ++m) {
      const T* const x = static_cast<const T*>(left) + m * left_ld;
      float top = 0.0f;
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        const int k = 8 * (threadIdx.x + h * blockDim.x);
        if (k < depth) {
          load8(x + k, depth - k, held[h]);
          top = fmaxf(top, magnitude8(held[h]));
        }
      }
      for (int k = 8 * (threadIdx.x + kHeld * blockDim.x); k < depth; k += 8 * blockDim.x) {
        load8(x + k, depth - k, v);
        top = fmaxf(top, magnitude8(v));
      }
      top = wave_max_magnitude(top);
      if (lane == 0) tops[m][wave] = top;
    }
    __syncthreads();
    for (int m = 0; m < rows; ++m) {
      const T* const x = static_cast<const T*>(left) + m * left_ld;
      float top = 0.0f, step;
      for (int i = 0; i < waves; ++i) top = fmaxf(top, tops[m][i]);
      const float inv = quantization(top, step);
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        const int k = 8 * (threadIdx.x + h * blockDim.x);
        if (k < pitch) {
          if (rows > 1 && k < depth) load8(x + k, depth - k, held[h]);
          store_levels(levels + m * pitch + k, 8, depth - k, held[h], inv);
        }
      }
      for (int k = 8 * (threadIdx.x + kHeld * blockDim.x); k < pitch; k += 8 * blockDim.x) {
        if (k < depth) load8(x + k, depth - k, v);
        store_levels(levels + m * pitch + k, 8, depth - k, v, inv);
      }
      if (threadIdx.x == 0) scales[m] = step;
    }
    __syncthreads();
    e.xs = scales;
  }
  const E* const lrow = QUANT ? nullptr : static_cast<const E*>(left) + lm * left_ld;
  auto load_left = [&](int k) {
    i32x4 v;
    if constexpr (QUANT)
      __builtin_memcpy(&v, __builtin_assume_aligned(levels + lm * pitch + k, 16), 16);
    else
      __builtin_memcpy(&v, lrow + k, 16);
    return v;
  };

  Acc acc = {};
  int s = s0;
  if (deep) {
    // each register of weights is refilled as soon as it is used
    i32x4 x[kDeep];
    for (; s + 2 * kDeep <= s1w; s += kDeep) {
#pragma unroll
      for (int j = 0; j < kDeep; ++j) x[j] = load_left((s + j) * kStep + k0);
#pragma unroll
      for (int j = 0; j < kDeep; ++j) {
        acc = M::mma(w[j], x[j], acc);
        __builtin_memcpy(&w[j], rrow + (s + kDeep + j) * kStep + k0, 16);
      }
    }
#pragma unroll
    for (int j = 0; j < kDeep; ++j) x[j] = load_left((s + j) * kStep + k0);
#pragma unroll
    for (int j = 0; j < kDeep; ++j) acc = M::mma(w[j], x[j], acc);
    s += kDeep;
  }
  for (; s < s1; ++s) {
    const int k = s * kStep + k0;
    i32x4 x = {0, 0, 0, 0};
    if constexpr (QUANT) {
      if (k < pitch) x = load_left(k);
    } else {
      x = load_chunk(lrow, k, depth);
    }
    acc = M::mma(load_chunk(rrow, k, depth), x, acc);
  }
  sums[wave][li][lane >> 4] = acc;
  if constexpr (ADAPT) {
    float* const s = reinterpret_cast<float*>(levels);
    const int count = rows * ad->pitch();
    if (static_cast<int>(threadIdx.x) < count) s[threadIdx.x] = held_s;
    for (int i = threadIdx.x + blockDim.x; i < count; i += blockDim.x) s[i] = adapter_sum(*ad, count, i);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < R * R; i += blockDim.x) {
    const int m = i / R, n = i % R;
    auto a = sums[0][m][n >> 2][n & 3];
    a = 0;
    for (int v = 0; v < waves; ++v)
#pragma unroll
      for (int g = 0; g < G; ++g) a += sums[v][g * R + m][(g * R + n) >> 2][n & 3];
    out[m][n] = static_cast<float>(a);
    if constexpr (ADAPT) {  // (as many threads as outputs: one step)
      if (brow != nullptr) {
        const float* const s = reinterpret_cast<const float*>(levels) + m * ad->pitch();
        float v = 0.0f;
#pragma unroll
        for (int c = 0; c < kHeldRank / 8; ++c)
          if (8 * c < ad->rank) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v += raw_element<T>(held_b[c], j) * s[8 * c + j];
          }
        for (int k = kHeldRank; k < ad->rank; k += 8) {
          const raw8 b = load_raw8<T, false>(brow, k, ad->rank - k);
#pragma unroll
          for (int j = 0; j < 8; ++j) v += raw_element<T>(b, j) * s[k + j];
        }
        out[m][n] += v;
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (R / 8); i += blockDim.x) {
    const int m = i / (R / 8), c = 8 * (i % (R / 8));
    if (n0 + c >= cols) continue;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = out[m][c + j];
    finish8<T, ACT, FULL>(v, e, m, n0 + c, cols);
  }
}

template <typename M, typename T, int R, bool QUANT, int ACT, bool FULL>
__global__ __launch_bounds__(64 * kFewWaves) void product_few_kernel(int rows, int cols, int depth, int per,
                                                                     const void* __restrict__ left, long left_ld,
                                                                     const typename M::elem* __restrict__ right,
                                                                     long right_ld, Epilogue e) {
  product_few<M, T, R, QUANT, ACT, FULL>(rows, cols, depth, per, left, left_ld, right, right_ld, e);
}

template <typename M, typename T, int R, int ACT, bool FULL>
__global__ __launch_bounds__(64 * kFewWaves) void product_few_adapters_kernel(int rows, int cols, int depth, int per,
                                                                              const void* __restrict__ left, long left_ld,
                                                                              const typename M::elem* __restrict__ right,
                                                                              long right_ld, Epilogue e, Adapters ad) {
  product_few<M, T, R, false, ACT, FULL, true>(rows, cols, depth, per, left, left_ld, right, right_ld, e, &ad);
}

template <typename M, typename T, int R, bool QUANT>
static hipError_t launch_few(const Product& pr, hipStream_t st) {
  typedef typename M::elem E;
  const int step = 16 / R * 64;
  const int steps = (pr.depth * static_cast<int>(sizeof(E)) + step - 1) / step;
  // eight steps a wave are all in flight at once; eight waves, so that several workgroups share
  // a CU and one's sums and epilogue overlap another's loads
  const int waves = steps >= 64 ? 8 : 4;
  const int per = (steps + waves - 1) / waves;
  const size_t lds = QUANT ? static_cast<size_t>(pr.rows) * ((pr.depth + 15) / 16 * 16) : 0;
  with_activation(pr.epi.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    const auto kernel = pr.cols % 8 == 0 ? product_few_kernel<M, T, R, QUANT, ACT, true> : product_few_kernel<M, T, R, QUANT, ACT, false>;
    hipLaunchKernelGGL(kernel, dim3((pr.cols + R - 1) / R), dim3(64 * waves), lds, st, pr.rows, pr.cols, pr.depth, per,
                       pr.left, pr.left_ld, static_cast<const E*>(pr.right), pr.right_ld, pr.epi);
  });
  return hipGetLastError();
}

// ---- products with adapters ---------------------------------------------------------------
template <typename M, typename T, int R>
static hipError_t launch_few_adapters(const Product& pr, const Adapters& ad, hipStream_t st) {
  typedef typename M::elem E;
  const int step = 16 / R * 64;
  const int steps = (pr.depth * static_cast<int>(sizeof(E)) + step - 1) / step;
  const int waves = steps >= 64 ? 8 : 4;  // as without adapters
  const int per = (steps + waves - 1) / waves;
  with_activation(pr.epi.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    const auto kernel = pr.cols % 8 == 0 ? product_few_adapters_kernel<M, T, R, ACT, true> : product_few_adapters_kernel<M, T, R, ACT, false>;
    hipLaunchKernelGGL(kernel, dim3((pr.cols + R - 1) / R), dim3(64 * waves), sizeof(float) * pr.rows * ad.pitch(), st, pr.rows,
                       pr.cols, pr.depth, per, pr.left, pr.left_ld, static_cast<const E*>(pr.right), pr.right_ld, pr.epi, ad);
  });
  return hipGetLastError();
}

template <typename M, typename T, typename S>
static hipError_t launch_tile_adapters(const Product& pr, const Adapters& ad, hipStream_t st) {
  typedef typename M::elem E;
  const int tiles_m = (pr.rows + S::BM - 1) / S::BM, tiles_n = (pr.cols + S::BN - 1) / S::BN;
  const int stages = (pr.depth * static_cast<int>(sizeof(E)) + kStageBytes - 1) / kStageBytes;
  auto launch = [&](auto kernel, int parts) {
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(tiles_m) * static_cast<unsigned>(tiles_n), parts), dim3(64 * S::WAVES), 0,
                       st, pr.rows, pr.cols, pr.depth, (stages + parts - 1) / parts, static_cast<const E*>(pr.left), pr.left_ld,
                       static_cast<const E*>(pr.right), pr.right_ld, pr.epi, static_cast<typename M::acc*>(pr.partial), tiles_m,
                       tiles_n, ad);
    return hipGetLastError();
  };
  if constexpr (S::BM < 256) {  // (a 256 x 256 tile's plan has one part)
    if (pr.plan.splits > 1) {
      const hipError_t err = launch(product_adapters_kernel<M, T, S, kOutPartial>, pr.plan.splits);
      return err != hipSuccess ? err : launch_join<M, T>(pr, st);
    }
  }
  return launch(product_adapters_kernel<M, T, S, kOutEpilogue>, 1);
}

template <typename M, typename T>
static hipError_t launch_adapters(const Product& pr, const Adapters& ad, hipStream_t st) {
  switch (pr.plan.tile) {
    case kFew8:
      return launch_few_adapters<M, T, 8>(pr, ad, st);
    case kFew16:
      return launch_few_adapters<M, T, 16>(pr, ad, st);
    case kTile256:
      return launch_tile_adapters<M, T, Tile256>(pr, ad, st);
    case kTile128:
      return launch_tile_adapters<M, T, Tile128>(pr, ad, st);
    case kTile128Deep:
      return launch_tile_adapters<M, T, Tile128Deep>(pr, ad, st);
    case kTile64:
      return launch_tile_adapters<M, T, Tile64>(pr, ad, st);
  }
  return hipErrorInvalidValue;
}

// Every product of one operand type.
template <typename M, typename T>
static hipError_t launch_type(const Product& pr, hipStream_t st) {
  if (!pr.left_along_index && !pr.right_along_index) {
    if (pr.plan.tile == kFew8 || pr.plan.tile == kFew16) {
      const bool eight = pr.plan.tile == kFew8;
      if constexpr (sizeof(typename M::elem) == 1) {
        if (pr.quantize) return eight ? launch_few<M, T, 8, true>(pr, st) : launch_few<M, T, 16, true>(pr, st);
      }
      return eight ? launch_few<M, T, 8, false>(pr, st) : launch_few<M, T, 16, false>(pr, st);
    }
    return launch_layout<M, T, kAlongDepth, kAlongDepth, kOutEpilogue>(pr, st);
  }
  if constexpr (sizeof(typename M::elem) == 2) {
    if (!pr.left_along_index) return launch_layout<M, T, kAlongDepth, kAlongIndex, kOutPlain>(pr, st);
    if (pr.right_along_index) return launch_layout<M, T, kAlongIndex, kAlongIndex, kOutPlain>(pr, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace oz2
