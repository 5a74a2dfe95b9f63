// oz2_norm_api.hip -- the norm's entry points declared in include/oz2.h: argument checks,
// workspace and launches on the caller's stream.
#include <cfloat>
#include <initializer_list>

#include "oz2_args.hpp"
#include "oz2_norm.hpp"

using namespace oz2::args;

namespace {

static_assert(OZ2_NORM_MAX_Q == oz2::kNormMaxCols, "the kernels' longest row");

bool eps_ok(double eps) { return eps >= FLT_MIN && eps <= 1e6; }  // (NaN is neither)

bool type_ok(int type) { return type >= OZ2_BF16 && type <= OZ2_F32; }

// What both forward calls check; OZ2_OK with nothing left to do where p or q is 0.
int check_norm(int type, int p, int q, const Mat& x, const Mat& res, const Mat& w, double eps, const Mat& h) {
  if (!type_ok(type) || !sizes_ok(p, q, 0) || !eps_ok(eps)) return OZ2_ERR_ARG;
  if (!ld_ok(x) || !ld_ok(res) || !ld_ok(h)) return OZ2_ERR_ARG;
  if (q > OZ2_NORM_MAX_Q) return OZ2_ERR_UNSUPPORTED;
  if (p > 0 && q > 0 && x.ptr == nullptr) return OZ2_ERR_ARG;
  if ((overlap(h, x) && !same(h, x)) || (overlap(h, res) && !same(h, res)) || overlap(h, w)) return OZ2_ERR_ARG;
  return OZ2_OK;
}

}  // namespace

extern "C" {

int ozaki2_rms_norm(int type, int p, int q, const void* X, int ldx, const void* R, int ldr, const void* w, double eps,
                    void* H, int ldh, void* Y, int ldy, void* stream) {
  const size_t e = elem_of(type);
  const Mat x{X, p, q, ldx, e}, res{R, p, q, ldr, e}, wm{w, 1, q, q, e}, h{H, p, q, ldh, e}, y{Y, p, q, ldy, e};
  const int rc = check_norm(type, p, q, x, res, wm, eps, h);
  if (rc != OZ2_OK) return rc;
  if (!ld_ok(y)) return OZ2_ERR_ARG;
  if (p == 0 || q == 0) return OZ2_OK;
  if (Y == nullptr) return OZ2_ERR_ARG;
  if ((overlap(y, x) && !same(y, x)) || (overlap(y, res) && !same(y, res)) || overlap(y, wm) || overlap(y, h)) return OZ2_ERR_ARG;
  return status(oz2::launch_rms_norm({type, p, q, X, ldx, R, ldr, w, static_cast<float>(eps), H, ldh, Y, ldy, nullptr, 0, nullptr},
                                     static_cast<hipStream_t>(stream)));
}

int ozaki2_rms_norm_i8(int type, int p, int q, const void* X, int ldx, const void* R, int ldr, const void* w, double eps,
                       void* H, int ldh, int8_t* Q, int ldq, float* scale, void* stream) {
  const size_t e = elem_of(type);
  const Mat x{X, p, q, ldx, e}, res{R, p, q, ldr, e}, wm{w, 1, q, q, e}, h{H, p, q, ldh, e}, out{Q, p, q, ldq, 1},
      sc{scale, 1, p, p, sizeof(float)};
  const int rc = check_norm(type, p, q, x, res, wm, eps, h);
  if (rc != OZ2_OK) return rc;
  if (!ld_ok(out)) return OZ2_ERR_ARG;
  if (p == 0) return OZ2_OK;
  if (scale == nullptr || (q > 0 && Q == nullptr)) return OZ2_ERR_ARG;
  for (const Mat* o : {&out, &sc})
    if (overlap(*o, x) || overlap(*o, res) || overlap(*o, wm) || overlap(*o, h)) return OZ2_ERR_ARG;
  if (overlap(sc, out)) return OZ2_ERR_ARG;
  return status(oz2::launch_rms_norm({type, p, q, X, ldx, R, ldr, w, static_cast<float>(eps), H, ldh, nullptr, 0, Q, ldq, scale},
                                     static_cast<hipStream_t>(stream)));
}

int ozaki2_rms_norm_bwd(int type, int p, int q, const void* dY, int lddy, const void* H, int ldh, const void* w, double eps,
                        const void* dH, int lddh, void* dX, int lddx, void* dw, void* work, size_t work_bytes, void* stream) {
  const size_t e = elem_of(type);
  const Mat dy{dY, p, q, lddy, e}, h{H, p, q, ldh, e}, wm{w, 1, q, q, e}, dh{dH, p, q, lddh, e}, dx{dX, p, q, lddx, e},
      dwm{dw, 1, q, q, e};
  if (!type_ok(type) || !sizes_ok(p, q, 0) || !eps_ok(eps)) return OZ2_ERR_ARG;
  if (!ld_ok(dy) || !ld_ok(h) || !ld_ok(dh) || !ld_ok(dx)) return OZ2_ERR_ARG;
  if (q > OZ2_NORM_MAX_Q) return OZ2_ERR_UNSUPPORTED;
  if (q == 0 || (dX == nullptr && dw == nullptr) || (p == 0 && dw == nullptr)) return OZ2_OK;
  if (p > 0 && (dY == nullptr || H == nullptr)) return OZ2_ERR_ARG;
  if ((overlap(dx, dy) && !same(dx, dy)) || (overlap(dx, dh) && !same(dx, dh)) || overlap(dx, h) || overlap(dx, wm)) return OZ2_ERR_ARG;
  for (const Mat* i : {&dy, &h, &wm, &dh, &dx})
    if (overlap(dwm, *i)) return OZ2_ERR_ARG;
  float* part = nullptr;
  const int rc = workspace(work, work_bytes, part, [&](Carver& c) {
    return dw == nullptr ? nullptr : static_cast<float*>(c.take(sizeof(float) * oz2::norm_grad_blocks(p, q) * q));
  });
  if (rc != OZ2_OK) return rc;
  return status(oz2::launch_rms_norm_bwd({type, p, q, dY, lddy, H, ldh, w, static_cast<float>(eps), dH, lddh, dX, lddx, dw, part},
                                         static_cast<hipStream_t>(stream)));
}

size_t ozaki2_rms_norm_bwd_workspace_size(int type, int p, int q) {
  if (!type_ok(type) || !sizes_ok(p, q, 0) || q > OZ2_NORM_MAX_Q) return 0;
  Carver c;
  c.take(sizeof(float) * oz2::norm_grad_blocks(p, q) * q);
  return c.used;
}

}  // extern "C"
