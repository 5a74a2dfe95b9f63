// oz2_logprobs_api.hip -- the entry points of tokens' log probabilities declared in include/oz2.h:
// argument checks, workspace and launches on the caller's stream.
#include "oz2_args.hpp"
#include "oz2_logprobs.hpp"

using namespace oz2::args;

namespace {

static_assert(OZ2_MAX_TOP == oz2::kMaxTop, "one of the largest per lane");

bool type_ok(int type) { return type >= OZ2_BF16 && type <= OZ2_F32; }

struct Work {
  float4* stats;
  uint64_t* keys;
};

Work carve(Carver& c, int p, int v, int top) {
  Work w{};
  const size_t parts = oz2::logprobs_parts(p, v);
  if (parts <= 1) return w;
  w.stats = static_cast<float4*>(c.take(sizeof(float4) * parts * p));
  if (top > 0) w.keys = static_cast<uint64_t*>(c.take(sizeof(uint64_t) * parts * p * top));
  return w;
}

Mat vec(const void* ptr, long n, size_t elem) { return {ptr, 1, n, n, elem}; }

}  // namespace

extern "C" {

int ozaki2_token_logprobs(int type, int p, int v, const void* L, int ldl, const int64_t* tokens, int top, float* logprob,
                          float* lse, float* entropy, int64_t* top_tokens, float* top_logprob, void* work,
                          size_t work_bytes, void* stream) {
  if (!type_ok(type) || !sizes_ok(p, v, 0) || top < 0 || top > OZ2_MAX_TOP || top > v) return OZ2_ERR_ARG;
  const Mat l{L, p, v, ldl, elem_of(type)}, tk = vec(tokens, p, 8);
  const Mat outs[] = {vec(logprob, p, 4), vec(lse, p, 4), vec(entropy, p, 4), vec(top_tokens, static_cast<long>(p) * top, 8),
                      vec(top_logprob, static_cast<long>(p) * top, 4)};
  if (!ld_ok(l)) return OZ2_ERR_ARG;
  if (p == 0) return OZ2_OK;
  if ((v > 0 && L == nullptr) || (logprob != nullptr && tokens == nullptr)) return OZ2_ERR_ARG;
  if (top > 0 && (top_tokens == nullptr || top_logprob == nullptr)) return OZ2_ERR_ARG;
  for (const Mat& o : outs) {
    if (overlap(o, l) || overlap(o, tk)) return OZ2_ERR_ARG;
    for (const Mat& o2 : outs)
      if (&o != &o2 && overlap(o, o2)) return OZ2_ERR_ARG;
  }
  Work ws;
  const int rc = workspace(work, work_bytes, ws, [&](Carver& c) { return carve(c, p, v, top); });
  if (rc != OZ2_OK) return rc;
  return status(oz2::launch_logprobs({type, p, v, L, ldl, tokens, top, logprob, lse, entropy, top_tokens, top_logprob, ws.stats, ws.keys},
                                     static_cast<hipStream_t>(stream)));
}

size_t ozaki2_token_logprobs_workspace_size(int p, int v, int top) {
  if (!sizes_ok(p, v, 0) || top < 0 || top > OZ2_MAX_TOP) return 0;
  Carver c;
  carve(c, p, v, top);
  return c.used;
}

int ozaki2_token_logprobs_bwd(int type, int p, int v, const float* dlogprob, const void* L, int ldl, const int64_t* tokens,
                              const float* lse, const float* dentropy, const float* entropy, void* dL, int lddl, void* stream) {
  if (!type_ok(type) || !sizes_ok(p, v, 0)) return OZ2_ERR_ARG;
  const size_t e = elem_of(type);
  const Mat l{L, p, v, ldl, e}, d{dL, p, v, lddl, e};
  if (!ld_ok(l) || !ld_ok(d)) return OZ2_ERR_ARG;
  if (p == 0 || v == 0) return OZ2_OK;
  if (L == nullptr || lse == nullptr || dL == nullptr) return OZ2_ERR_ARG;
  if ((dlogprob != nullptr && tokens == nullptr) || (dentropy != nullptr && entropy == nullptr)) return OZ2_ERR_ARG;
  if (overlap(d, l) && !same(d, l)) return OZ2_ERR_ARG;
  for (const Mat& i : {vec(dlogprob, p, 4), vec(tokens, p, 8), vec(lse, p, 4), vec(dentropy, p, 4), vec(entropy, p, 4)})
    if (overlap(d, i)) return OZ2_ERR_ARG;
  return status(oz2::launch_logprobs_bwd({type, p, v, dlogprob, L, ldl, tokens, lse, dentropy, entropy, dL, lddl},
                                         static_cast<hipStream_t>(stream)));
}

}  // extern "C"
