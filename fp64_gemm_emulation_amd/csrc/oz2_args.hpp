// oz2_args.hpp -- what the entry points on row-major matrices share: their checks of arguments
// and the layout of a call's workspace.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "oz2.h"
#include "oz2_internal.hpp"

namespace oz2::args {

constexpr size_t kAlign = 256;
constexpr long kMaxDim = 1L << 23;  // as for the FP64 products

// One matrix argument: rows x cols elements, row stride ld.
struct Mat {
  const void* ptr;
  long rows, cols, ld;
  size_t elem;
  bool empty() const { return ptr == nullptr || rows == 0 || cols == 0; }
  size_t bytes() const { return elem * (static_cast<size_t>(ld) * (rows - 1) + cols); }
};

// Whether two matrices share an element: their address ranges meet, and, where their rows have
// the same stride, so do the columns they take of it (two column ranges of one wide buffer are
// apart although their address ranges interleave).
inline bool overlap(const Mat& a, const Mat& b) {
  if (a.empty() || b.empty()) return false;
  const auto pa = reinterpret_cast<uintptr_t>(a.ptr), pb = reinterpret_cast<uintptr_t>(b.ptr);
  if (pa >= pb + b.bytes() || pb >= pa + a.bytes()) return false;
  const size_t pitch = a.elem * a.ld;
  if (pitch != b.elem * b.ld) return true;
  const size_t d = pb >= pa ? (pb - pa) % pitch : (pitch - (pa - pb) % pitch) % pitch;
  return d < a.elem * a.cols || d + b.elem * b.cols > pitch;
}

inline bool same(const Mat& a, const Mat& b) { return a.ptr == b.ptr && a.ld == b.ld; }

inline bool sizes_ok(int p, int q, int r) {
  return p >= 0 && q >= 0 && r >= 0 && p <= kMaxDim && q <= kMaxDim && r <= kMaxDim;
}

inline bool ld_ok(const Mat& m) { return m.ptr == nullptr || m.ld >= std::max(1L, m.cols); }

inline size_t elem_of(int type) { return type == OZ2_F32 ? 4 : 2; }

// Workspace: consecutive aligned pieces of `base` (null while only the size is asked for).
struct Carver {
  char* base = nullptr;
  size_t used = 0;
  void* take(size_t bytes) {
    void* const p = base != nullptr ? base + used : nullptr;
    used += (bytes + kAlign - 1) / kAlign * kAlign;
    return p;
  }
};

// Lays out the call's workspace, carve(carver), in the caller's memory if given, else in the
// library's (where the size has to be known first).
template <typename Work, typename F>
int workspace(void* work, size_t work_bytes, Work& ws, F carve) {
  if (reinterpret_cast<uintptr_t>(work) % kAlign != 0) return OZ2_ERR_ARG;
  Carver c{static_cast<char*>(work)};
  ws = carve(c);
  if (work != nullptr) return work_bytes < c.used ? OZ2_ERR_WORKSPACE : OZ2_OK;
  if (c.used == 0) return OZ2_OK;
  Carver owned;
  const int rc = oz2::acquire_linear_workspace(c.used, &owned.base);
  if (rc == OZ2_OK) ws = carve(owned);
  return rc;
}

inline int status(hipError_t e) { return e == hipSuccess ? OZ2_OK : OZ2_ERR_HIP; }

}  // namespace oz2::args
