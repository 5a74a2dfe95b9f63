// oz2_logprobs.hpp -- launch interface of the log probabilities of tokens between
// oz2_logprobs_api.hip and the kernels in oz2_logprobs.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace oz2 {

constexpr int kMaxTop = 64;  // one per lane of a wave

struct Logprobs {
  int type, p, v;
  const void* logits;
  long ld;
  const int64_t* tokens;  // null: no logprob
  int top;
  float *logprob, *lse, *entropy;  // each may be null
  int64_t* top_tokens;
  float* top_logprob;
  // where a row is read by several workgroups: four floats for each, and `top` keys
  float4* stats;
  uint64_t* keys;
};
// Workgroups that share a row.
int logprobs_parts(int p, int v);
hipError_t launch_logprobs(const Logprobs& l, hipStream_t st);

struct LogprobsGrad {
  int type, p, v;
  const float* dlogprob;  // null: none
  const void* logits;
  long ld;
  const int64_t* tokens;
  const float* lse;
  const float *dentropy, *entropy;  // null: none
  void* dlogits;  // may be logits
  long ldd;
};
hipError_t launch_logprobs_bwd(const LogprobsGrad& l, hipStream_t st);

}  // namespace oz2
