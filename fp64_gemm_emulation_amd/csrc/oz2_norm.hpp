// oz2_norm.hpp -- launch interface of the root-mean-square norm between oz2_norm_api.hip and the
// kernels in oz2_norm.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace oz2 {

// Longest row: 1024 threads hold 32 elements each.
constexpr int kNormMaxCols = 32768;

// Rows of h = x + res (rounded to the type; res null: h = x) times (mean(h^2) + eps)^(-1/2) times
// w (null: ones).  h is stored where h is not null; the result goes to y, or, where y is null, as
// int8 levels with one scale per row.
struct Norm {
  int type, p, q;
  const void* x;
  long ldx;
  const void* res;
  long ldr;
  const void* w;
  float eps;
  void* h;
  long ldh;
  void* y;
  long ldy;
  int8_t* levels;
  long ldl;
  float* scale;
};
hipError_t launch_rms_norm(const Norm& n, hipStream_t st);

// dx = the norm's gradient from dy and h, plus dh (null: none); dw (null: not computed) by way of
// part: norm_grad_blocks(p, q) rows of q floats.
struct NormGrad {
  int type, p, q;
  const void* dy;
  long lddy;
  const void* h;
  long ldh;
  const void* w;
  float eps;
  const void* dh;
  long lddh;
  void* dx;
  long lddx;
  void* dw;
  float* part;
};
int norm_grad_blocks(int p, int q);
hipError_t launch_rms_norm_bwd(const NormGrad& n, hipStream_t st);

}  // namespace oz2
