// oz2_logprobs.hip -- log probabilities of given tokens from rows of logits, with the rows'
// entropy and their largest log probabilities, and the logits' gradient.
#include <algorithm>
#include <cfloat>

#include "oz2_common.hpp"
#include "oz2_linear.hpp"
#include "oz2_logprobs.hpp"

namespace oz2 {

// Matrices above this are read and written with the non-temporal hint: with their like they
// exceed the 256 MB memory-side cache.
constexpr double kStreamBytes = 64.0 * (1 << 20);
constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
// exp of this is 0 in f32, and 0 times it 0: what a difference of logits is held above where it
// is a factor, as 0 times the -Inf of a masked logit would be NaN
constexpr float kGone = -200.0f;

__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

// Softmax statistics of a set of logits: its maximum m (at least -FLT_MAX, so that differences
// from it are defined), s = sum exp(l - m) and t = sum exp(l - m) (l - m).  A NaN or +Inf among
// the logits makes s NaN.
struct Stats {
  float m, s, t;
  static __device__ __forceinline__ Stats none() { return {-FLT_MAX, 0.0f, 0.0f}; }
  __device__ __forceinline__ void raise(float to) {
    const float d = fmaxf(m - to, kGone), f = exp_of(d);
    t = f * __builtin_fmaf(d, s, t);
    s *= f;
    m = to;
  }
  __device__ __forceinline__ void join(const Stats& o) {
    Stats b = o;
    const float to = fmaxf(m, b.m);
    raise(to);
    b.raise(to);
    s += b.s;
    t += b.t;
  }
};

template <bool ENTROPY>
__device__ __forceinline__ void add8(Stats& a, const float (&l)[8]) {
  OZ2_UNROLL
  for (int i = 0; i < 8; ++i) {
    const float d = l[i] - a.m, e = exp_of(d);
    a.s += e;
    if constexpr (ENTROPY) a.t = __builtin_fmaf(e, fmaxf(d, kGone), a.t);
  }
}

__device__ __forceinline__ float max8(const float (&l)[8]) {  // (NaN is left out)
  return fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), fmaxf(fmaxf(l[4], l[5]), fmaxf(l[6], l[7])));
}

__device__ __forceinline__ Stats wave_join(Stats a) {
  OZ2_UNROLL
  for (int off = 32; off > 0; off >>= 1) {
    Stats b;
    b.m = __shfl_xor(a.m, off, 64);
    b.s = __shfl_xor(a.s, off, 64);
    b.t = __shfl_xor(a.t, off, 64);
    a.join(b);
  }
  return a;
}

// ---- the largest logits -------------------------------------------------------------------
// Keys: the value's order in the upper half, the negated index in the lower, so that keys are
// distinct, larger values come first and of equal ones the lowest index.  -0 is 0 and NaN is -Inf.
// 0 is below every key.
__device__ __forceinline__ uint32_t order_of(float l) {
  l = l != l ? -__builtin_inff() : l + 0.0f;
  const uint32_t b = __builtin_bit_cast(uint32_t, l);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __builtin_bit_cast(float, o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float l, uint32_t index) {
  return static_cast<uint64_t>(order_of(l)) << 32 | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ int64_t index_of(uint64_t key) { return 0xFFFFFFFFu - static_cast<uint32_t>(key); }

// Lane l's value from lane l ^ MASK: within rows of 16 lanes by data-parallel primitives, whose
// latency is a few cycles where a permute through LDS takes some 60 (a sort of 64 keys has 18 of its 21
// exchanges there).
template <int MASK>
__device__ __forceinline__ uint32_t lane_xor32(uint32_t v) {
  constexpr int kQuad1 = 0xB1, kQuad2 = 0x4E, kQuad3 = 0x1B, kMirror = 0x140, kHalfMirror = 0x141;  // xor 1, 2, 3, 15, 7
  auto dpp = [](uint32_t x, auto ctrl) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  if constexpr (MASK == 1) return dpp(v, std::integral_constant<int, kQuad1>{});
  else if constexpr (MASK == 2) return dpp(v, std::integral_constant<int, kQuad2>{});
  else if constexpr (MASK == 4) return dpp(dpp(v, std::integral_constant<int, kHalfMirror>{}), std::integral_constant<int, kQuad3>{});
  else if constexpr (MASK == 8) return dpp(dpp(v, std::integral_constant<int, kMirror>{}), std::integral_constant<int, kHalfMirror>{});
  else return __shfl_xor(v, MASK, 64);
}
template <int MASK>
__device__ __forceinline__ uint64_t lane_xor(uint64_t v) {
  return static_cast<uint64_t>(lane_xor32<MASK>(static_cast<uint32_t>(v >> 32))) << 32 | lane_xor32<MASK>(static_cast<uint32_t>(v));
}
template <int J>
__device__ __forceinline__ uint64_t exchange(uint64_t v, bool larger) {
  const uint64_t o = lane_xor<J>(v);
  return (v > o) == larger ? v : o;
}
// Exchanges at distances J, J / 2, ... 1; falls: whether the lane's run of 2 J is to fall.
template <int J>
__device__ __forceinline__ uint64_t exchanges(uint64_t v, bool falls) {
  v = exchange<J>(v, ((threadIdx.x & J) == 0) == falls);
  if constexpr (J > 1) v = exchanges<J / 2>(v, falls);
  return v;
}
// One key per lane, into falling order (a bitonic sorting network).
template <int K = 2>
__device__ __forceinline__ uint64_t wave_sort(uint64_t v) {
  v = exchanges<K / 2>(v, (threadIdx.x & K) == 0 || K == 64);
  if constexpr (K < 64) v = wave_sort<2 * K>(v);
  return v;
}
// The 64 largest of two sorted waves, sorted.
__device__ __forceinline__ uint64_t wave_merge(uint64_t a, uint64_t b) {
  b = lane_xor<63>(b);  // b in rising order
  return exchanges<32>(a > b ? a : b, true);
}
// The 64 largest over the workgroup's sorted waves, sorted, in best[0 .. 63].
template <int WAVES>
__device__ __forceinline__ void group_top(uint64_t sorted, uint64_t (&best)[WAVES][64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
  best[wave][lane] = sorted;
#pragma unroll 1
  for (int n = WAVES / 2; n > 0; n /= 2) {
    __syncthreads();
    if (wave < n && best[wave + n][0] != 0) best[wave][lane] = wave_merge(best[wave][lane], best[wave + n][lane]);
  }
  __syncthreads();
}

constexpr int kUnroll = 4;   // chunks of eight logits a thread has under way
constexpr int kList = 1024;  // candidates held at a time

// Eight logits of a chunk, -Inf beyond the row's end.
template <typename T, bool NT>
__device__ __forceinline__ void load_logits(const T* row, int chunk, int v, float (&l)[8]) {
  const int valid = v - 8 * chunk;
  load8<T, NT>(row + 8 * static_cast<long>(chunk), valid, l);
  if (valid < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= valid) l[i] = -__builtin_inff();
  }
}

struct Top {
  uint64_t best[kWaves][64];
  uint64_t bounds[kWaves];
  uint64_t list[kList];
  unsigned count;
};

// The `top` largest logits of chunks c0 .. c1 - 1 of a row as sorted keys, in s.best[0]; a thread
// has read every kThreads-th chunk from c0 + threadIdx.x on, and found its largest logit `most`
// first in chunk `at` (negative: no chunk).  The top-th largest of the threads' maxima, of all or of
// one wave's, bounds the top-th largest logit from below; only the threads whose maximum reaches it
// look at their chunks again (from a cache), and collect what reaches it: a few times `top` of
// independent logits.  Where there are more than the list holds (rows in rising order, a few runs of large
// ones), the top-th largest of the 1024 collected is a better bound: at least 1024 - top of them
// fall out, so the rounds end.
template <typename T>
__device__ __forceinline__ void top_of_chunks(Top& s, const T* row, int v, int c0, int c1, float most, int at, int top) {
  const uint64_t mine = at < 0 ? 0 : key_of(most, 8u * static_cast<unsigned>(at));  // no key of this thread is above
  uint64_t bound;
  if (top <= 32) {
    const uint64_t sorted = wave_sort(mine);
    if (static_cast<int>(threadIdx.x & 63) == top - 1) s.bounds[threadIdx.x >> 6] = sorted;
    __syncthreads();
    bound = s.bounds[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) bound = bound > s.bounds[w] ? bound : s.bounds[w];
  } else {  // (the least of a wave's 64 maxima would let too many through)
    group_top(wave_sort(mine), s.best);
    bound = s.best[0][top - 1];
  }
  // (the maximum may be any of its chunk's eight)
  bound = bound == 0 ? 1 : bound - 7;
  while (true) {
    if (threadIdx.x == 0) s.count = 0;
    __syncthreads();
    if (mine >= bound) {
      for (int c = c0 + static_cast<int>(threadIdx.x); c < c1; c += kThreads) {
        float l[8];
        load_logits<T, false>(row, c, v, l);
        if (key_of(max8(l), 8u * c) < bound) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t key = key_of(l[i], 8u * c + i);
          if (key < bound || 8 * c + i >= v) continue;
          const unsigned n = atomicAdd(&s.count, 1u);
          if (n < kList) s.list[n] = key;
        }
      }
    }
    __syncthreads();
    const unsigned found = s.count, held = min(found, static_cast<unsigned>(kList));
    uint64_t sorted = 0;
    for (unsigned n = 0; n < held; n += kThreads) {
      const uint64_t next = wave_sort(n + threadIdx.x < held ? s.list[n + threadIdx.x] : 0);
      sorted = n == 0 ? next : wave_merge(sorted, next);
    }
    group_top(sorted, s.best);
    if (found <= kList) return;
    bound = s.best[0][top - 1];
  }
}

// A row's results from its statistics and keys, by the workgroup's first wave.
template <typename T>
__device__ __forceinline__ void finish_row(const Logprobs& a, long row, const Stats& s, const uint64_t* keys) {
  const int lane = threadIdx.x;
  if (lane >= 64) return;
  // (l - m) - log s rather than l - lse: where the logits are large lse has lost log s
  const float logs = __builtin_amdgcn_logf(s.s) * kLn2;
  const bool none = s.s == 0.0f;  // every logit is -Inf
  auto logprob = [&](float l) { return none ? -__builtin_inff() : l - s.m - logs; };
  if (lane == 0) {
    if (a.lse != nullptr) a.lse[row] = none ? -__builtin_inff() : s.m + logs;
    if (a.entropy != nullptr) a.entropy[row] = none ? 0.0f : logs - s.t / s.s;
    if (a.logprob != nullptr) {
      const int64_t t = a.tokens[row];
      a.logprob[row] = t < 0 ? 0.0f
                       : t >= a.v ? __builtin_nanf("")
                                  : logprob(static_cast<float>(static_cast<const T*>(a.logits)[row * a.ld + t]));
    }
  }
  if (lane < a.top) {
    a.top_tokens[row * a.top + lane] = index_of(keys[lane]);
    a.top_logprob[row * a.top + lane] = logprob(value_of(keys[lane]));
  }
}

// One row, or the part blockIdx.y of it, per workgroup: one pass with running maximum and sums, which
// a step of 32 logits moves to its maximum at once.  Bound by memory: 4096 x 131072 bf16 with the
// entropy in 167 us, 6.4 TB/s (non-temporal loads).  16 rows of 131072 with 20 of the largest, in 32
// parts, take 9.2 to 9.4 us, of which the selection is about half, and the join 4.2.  The threads that look again
// have 16 bytes of nearly every line, so of many rows most is read twice: 4096 x 131072 with 1, 20 and 64
// of the largest 258, 388 and 394 us (174 with none on that board).
template <typename T, bool ENTROPY, bool TOP, bool NT>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(Logprobs a, int per) {
  __shared__ Stats waves[kWaves];
  __shared__ Top top;
  const long row = blockIdx.x;
  const T* const l = static_cast<const T*>(a.logits) + row * a.ld;
  const int chunks = (a.v + 7) / 8, c0 = per * static_cast<int>(blockIdx.y), c1 = min(c0 + per, chunks);
  const int whole = min(c1, a.v / 8);  // chunks before this one are full
  Stats s = Stats::none();
  float most = -__builtin_inff();
  int at = c0 + static_cast<int>(threadIdx.x) < c1 ? c0 + static_cast<int>(threadIdx.x) : -1;
  auto see = [&](const float (&x)[8], int c) {
    const float m = max8(x);
    if constexpr (TOP) {
      at = m > most ? c : at;
      most = fmaxf(m, most);
    }
    return m;
  };
  int c = c0 + static_cast<int>(threadIdx.x);
  for (; c + (kUnroll - 1) * kThreads < whole; c += kUnroll * kThreads) {
    float x[kUnroll][8], m = s.m;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) load8<T, NT>(l + 8 * static_cast<long>(c + u * kThreads), 8, x[u]);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) m = fmaxf(m, see(x[u], c + u * kThreads));
    s.raise(m);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) add8<ENTROPY>(s, x[u]);
  }
  for (; c < c1; c += kThreads) {
    float x[8];
    load_logits<T, NT>(l, c, a.v, x);
    s.raise(fmaxf(s.m, see(x, c)));
    add8<ENTROPY>(s, x);
  }
  s = wave_join(s);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = s;
  __syncthreads();
  s = waves[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s.join(waves[w]);
  if constexpr (TOP) top_of_chunks(top, l, a.v, c0, c1, most, at, a.top);
  if (gridDim.y == 1) {
    finish_row<T>(a, row, s, TOP ? top.best[0] : nullptr);
    return;
  }
  const long part = row * gridDim.y + blockIdx.y;
  if (threadIdx.x == 0) a.stats[part] = float4{s.m, s.s, s.t, 0.0f};
  if constexpr (TOP) {
    if (static_cast<int>(threadIdx.x) < a.top) a.keys[part * a.top + threadIdx.x] = top.best[0][threadIdx.x];
  }
}

// The parts of a row, joined in their order; every wave merges the sorted keys of some parts.
constexpr int kMaxParts = 64, kJoinWaves = 16;

template <typename T>
__global__ __launch_bounds__(64 * kJoinWaves) void logprobs_join_kernel(Logprobs a, int parts) {
  __shared__ uint64_t best[kJoinWaves][64];
  const long row = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Stats s = Stats::none();
  if (lane < parts && wave == 0) {
    const float4 f = a.stats[row * parts + lane];
    s.m = f.x;
    s.s = f.y;
    s.t = f.z;
  }
  if (a.top > 0) {
    const uint64_t* const keys = a.keys + row * parts * a.top;
    uint64_t own[kMaxParts / kJoinWaves];
#pragma unroll
    for (int i = 0; i < kMaxParts / kJoinWaves; ++i) {
      const int part = wave + kJoinWaves * i;
      own[i] = part < parts && lane < a.top ? keys[part * a.top + lane] : 0;
    }
#pragma unroll
    for (int i = 1; i < kMaxParts / kJoinWaves; ++i)
      if (wave + kJoinWaves * i < parts) own[0] = wave_merge(own[0], own[i]);
    group_top(own[0], best);
  }
  if (wave == 0) finish_row<T>(a, row, wave_join(s), best[0]);
}

// Few rows are divided among about 1024 workgroups (fewer than 1024 + p), with two chunks per thread and
// more but for a row's last part.
int logprobs_parts(int p, int v) {
  const int chunks = (v + 7) / 8;
  if (p <= 0 || chunks <= 2 * kThreads) return 1;
  const int wanted = std::min({(1024 + p - 1) / p, chunks / (2 * kThreads), kMaxParts});
  const int per = (chunks + std::max(wanted, 1) - 1) / std::max(wanted, 1);
  return (chunks + per - 1) / per;  // none of them empty
}

template <typename T>
static hipError_t logprobs(const Logprobs& a, hipStream_t st) {
  const int parts = logprobs_parts(a.p, a.v), per = ((a.v + 7) / 8 + parts - 1) / parts;
  const bool nt = static_cast<double>(a.p) * a.v * sizeof(T) > kStreamBytes;
  auto launch = [&](auto entropy, auto top) {
    constexpr bool E = decltype(entropy)::value, K = decltype(top)::value;
    const auto kernel = nt ? logprobs_kernel<T, E, K, true> : logprobs_kernel<T, E, K, false>;
    hipLaunchKernelGGL(kernel, dim3(a.p, parts), dim3(kThreads), 0, st, a, per);
  };
  if (a.entropy != nullptr)
    a.top > 0 ? launch(std::true_type{}, std::true_type{}) : launch(std::true_type{}, std::false_type{});
  else
    a.top > 0 ? launch(std::false_type{}, std::true_type{}) : launch(std::false_type{}, std::false_type{});
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || parts == 1) return err;
  hipLaunchKernelGGL(logprobs_join_kernel<T>, dim3(a.p), dim3(a.top > 0 ? 64 * kJoinWaves : 64), 0, st, a, parts);
  return hipGetLastError();
}

hipError_t launch_logprobs(const Logprobs& a, hipStream_t st) {
  if (a.type == kTypeBf16) return logprobs<bf16>(a, st);
  return a.type == kTypeF16 ? logprobs<f16>(a, st) : logprobs<float>(a, st);
}

// ---- gradient ------------------------------------------------------------------------------
// With p = exp(l - lse): dl = dlogprob (delta_token - p) - dentropy p (log p + entropy).
// lse is held in f32, so p is off by |lse| 2^-24: beyond kLseHeld (and where it is not finite) the
// workgroup works the row's maximum and sum out anew, and takes (l - m) - log s.
// Each of a row's workgroups reads all of it for that: 16 x 131072 bf16 24 us instead of 3.8, 4096 x 131072
// 511 instead of 404.  Below, exp(l - lse) is within 2^-18 of itself.
constexpr float kLseHeld = 64.0f;

// Bound by memory: 4096 x 131072 bf16, read and written once, in 400 us, 5.4 TB/s (the runtime's copy
// moves 5.1 both ways).
template <typename T, bool NT>
__global__ __launch_bounds__(kThreads) void logprobs_bwd_kernel(LogprobsGrad a, int per) {
  __shared__ Stats waves[kWaves];
  const long row = blockIdx.x;
  const T* const l = static_cast<const T*>(a.logits) + row * a.ld;
  T* const d = static_cast<T*>(a.dlogits) + row * a.ldd;
  const int chunks = (a.v + 7) / 8, c0 = per * static_cast<int>(blockIdx.y), c1 = min(c0 + per, chunks);
  float dlp = 0.0f;
  int token = -1;
  const float dh = a.dentropy != nullptr ? a.dentropy[row] : 0.0f;
  bool reached = dh != 0.0f;
  if (a.dlogprob != nullptr) {
    const int64_t t = a.tokens[row];
    dlp = t < 0 ? 0.0f : t >= a.v ? __builtin_nanf("") : a.dlogprob[row];
    token = t >= 0 && t < a.v ? static_cast<int>(t) : -1;
    reached = reached || t >= 0;
  }
  if (!reached) {  // whatever a padded place holds is not looked at
    const float zeros[8] = {};
    for (int c = c0 + static_cast<int>(threadIdx.x); c < c1; c += kThreads)
      store8<T, NT>(d + 8 * static_cast<long>(c), a.v - 8 * c, zeros);
    return;
  }
  float m = a.lse[row], logs = 0.0f;
  bool none = false;  // every logit is -Inf: no gradient
  if (!(fabsf(m) <= kLseHeld)) {
    Stats s = Stats::none();
    for (int c = threadIdx.x; c < chunks; c += kThreads) {
      float x[8];
      load_logits<T, false>(l, c, a.v, x);
      s.raise(fmaxf(s.m, max8(x)));
      add8<false>(s, x);
    }
    s = wave_join(s);
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = s;
    __syncthreads();
    s = waves[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s.join(waves[w]);
    // (every logit -Inf: a maximum above them leaves p = 0)
    none = s.s == 0.0f;
    m = none ? FLT_MAX : s.m;
    logs = none ? 0.0f : __builtin_amdgcn_logf(s.s) * kLn2;
  }
  // dlogprob + dentropy entropy (an entropy whose gradient is 0 is left out: it may not be finite)
  const float rest = dh == 0.0f ? dlp : __builtin_fmaf(dh, a.entropy[row] - logs, dlp);
  const float logs2 = logs * kLog2e;
  if (none) dlp = 0.0f;
  auto gradient = [&](float (&x)[8], int c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = x[i] - m, p = __builtin_amdgcn_exp2f(__builtin_fmaf(d, kLog2e, -logs2));
      x[i] = -p * __builtin_fmaf(dh, fmaxf(d, kGone), rest);
    }
    if (c == token >> 3) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] += i == (token & 7) ? dlp : 0.0f;
    }
  };
  int c = c0 + static_cast<int>(threadIdx.x);
  const int whole = min(c1, a.v / 8);
  for (; c + (kUnroll - 1) * kThreads < whole; c += kUnroll * kThreads) {
    float x[kUnroll][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) load8<T, NT>(l + 8 * static_cast<long>(c + u * kThreads), 8, x[u]);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      gradient(x[u], c + u * kThreads);
      store8<T, NT>(d + 8 * static_cast<long>(c + u * kThreads), 8, x[u]);
    }
  }
  for (; c < c1; c += kThreads) {
    float x[8];
    load_logits<T, NT>(l, c, a.v, x);
    gradient(x, c);
    store8<T, NT>(d + 8 * static_cast<long>(c), a.v - 8 * c, x);
  }
}

template <typename T>
static hipError_t logprobs_bwd(const LogprobsGrad& a, hipStream_t st) {
  // in place a row stays with one workgroup, which may have to read all of it first (16 x 131072 bf16 in 18 us,
  // 3.8 beside the logits)
  const int parts = a.dlogits == a.logits ? 1 : logprobs_parts(a.p, a.v), per = ((a.v + 7) / 8 + parts - 1) / parts;
  const bool nt = static_cast<double>(a.p) * a.v * sizeof(T) > kStreamBytes;
  const auto kernel = nt ? logprobs_bwd_kernel<T, true> : logprobs_bwd_kernel<T, false>;
  hipLaunchKernelGGL(kernel, dim3(a.p, parts), dim3(kThreads), 0, st, a, per);
  return hipGetLastError();
}

hipError_t launch_logprobs_bwd(const LogprobsGrad& a, hipStream_t st) {
  if (a.type == kTypeBf16) return logprobs_bwd<bf16>(a, st);
  return a.type == kTypeF16 ? logprobs_bwd<f16>(a, st) : logprobs_bwd<float>(a, st);
}

}  // namespace oz2
