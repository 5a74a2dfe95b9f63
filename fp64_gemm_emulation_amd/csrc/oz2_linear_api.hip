// oz2_linear_api.hip -- the linear-layer entry points declared in include/oz2.h: argument
// checks, workspace layout and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "oz2.h"
#include "oz2_internal.hpp"
#include "oz2_linear.hpp"

namespace {

constexpr size_t kAlign = 256;
constexpr long kMaxDim = 1L << 23;  // as for the FP64 products

static_assert(OZ2_BF16 == oz2::kTypeBf16 && OZ2_F16 == oz2::kTypeF16 && OZ2_F32 == oz2::kTypeF32, "types");
static_assert(OZ2_ACT_RELU == oz2::kActRelu && OZ2_ACT_GELU == oz2::kActGelu &&
                  OZ2_ACT_GELU_TANH == oz2::kActGeluTanh && OZ2_ACT_SILU == oz2::kActSilu,
              "activations");

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
bool overlap(const Mat& a, const Mat& b) {
  if (a.empty() || b.empty()) return false;
  const auto pa = reinterpret_cast<uintptr_t>(a.ptr), pb = reinterpret_cast<uintptr_t>(b.ptr);
  if (pa >= pb + b.bytes() || pb >= pa + a.bytes()) return false;
  const size_t pitch = a.elem * a.ld;
  if (pitch != b.elem * b.ld) return true;
  const size_t d = pb >= pa ? (pb - pa) % pitch : (pitch - (pa - pb) % pitch) % pitch;
  return d < a.elem * a.cols || d + b.elem * b.cols > pitch;
}

bool same(const Mat& a, const Mat& b) { return a.ptr == b.ptr && a.ld == b.ld; }

bool sizes_ok(int p, int q, int r) {
  return p >= 0 && q >= 0 && r >= 0 && p <= kMaxDim && q <= kMaxDim && r <= kMaxDim;
}

bool ld_ok(const Mat& m) { return m.ptr == nullptr || m.ld >= std::max(1L, m.cols); }

// One launch puts every 128 x 128 output tile along grid x (256 work-items each): that work-item
// count has to stay in 32 bits.
bool grid_ok(long rows, long cols) {
  return static_cast<uint64_t>((rows + 127) / 128) * static_cast<uint64_t>((cols + 127) / 128) * 256u < (1ull << 32);
}

size_t elem_of(int type) { return type == OZ2_F32 ? 4 : 2; }

bool drop_ok(const oz2_dropout_t* d) { return d == nullptr || (d->probability >= 0.0 && d->probability <= 1.0); }

oz2::Drop make_drop(const oz2_dropout_t* d) {
  oz2::Drop o;
  if (d == nullptr) return o;
  o.t = static_cast<uint32_t>(std::nearbyint(d->probability * 65536.0));
  o.scale = o.t < 65536u ? 65536.0f / static_cast<float>(65536u - o.t) : 0.0f;
  o.k0 = static_cast<uint32_t>(d->seed);
  o.k1 = static_cast<uint32_t>(d->seed >> 32);
  o.c2 = static_cast<uint32_t>(d->offset);
  o.c3 = static_cast<uint32_t>(d->offset >> 32);
  return o;
}

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

// The workspace of each call: copies of operands that need packing, and what it makes itself.
struct FwdWork {
  oz2::Plan plan;
  void *x, *w, *partial;
};

FwdWork carve_fwd(Carver& c, long p, long q, long r, bool pack_x, bool pack_w) {
  FwdWork w{};
  w.plan = oz2::plan_product(false, p, r, q, false, false);
  if (oz2::few_rows(w.plan)) return w;  // takes any rows
  if (pack_x) w.x = c.take(2 * p * oz2::packed_ld(q, 2));
  if (pack_w) w.w = c.take(2 * r * oz2::packed_ld(q, 2));
  w.partial = c.take(oz2::partial_bytes(w.plan, p, r));
  return w;
}

struct BwdWork {
  bool paired;  // both products in one launch
  oz2::Plan dx, dw;
  void *dz, *x, *w, *partial_x, *partial_w;
  float* sums;
};

BwdWork carve_bwd(Carver& c, long p, long q, long r, bool both, bool make_dz, bool pack_x, bool pack_w) {
  BwdWork w{};
  w.paired = both && oz2::plan_pair(p, q, r, w.dx, w.dw);
  if (!w.paired) {
    w.dx = oz2::plan_product(false, p, q, r, false, true);
    w.dw = oz2::plan_product(false, r, q, p, true, true);
  }
  if (make_dz) w.dz = c.take(2 * p * oz2::packed_ld(r, 2));
  if (pack_x) w.x = c.take(2 * p * oz2::packed_ld(q, 2));
  if (pack_w) w.w = c.take(2 * r * oz2::packed_ld(q, 2));
  w.partial_x = c.take(oz2::partial_bytes(w.dx, p, q));
  w.partial_w = c.take(oz2::partial_bytes(w.dw, r, q));
  w.sums = static_cast<float*>(c.take(sizeof(float) * oz2::grad_row_blocks(static_cast<int>(p), static_cast<int>(r)) * r));
  return w;
}

struct I8Work {
  oz2::Plan plan;
  int8_t *q, *v;
  float* scale;
  void* partial;
};

I8Work carve_i8(Carver& c, long p, long q, long r, bool pack_v) {
  I8Work w{};
  w.plan = oz2::plan_product(true, p, r, q, false, false);
  if (oz2::quantize_in_product(w.plan, p, q)) return w;
  w.q = static_cast<int8_t*>(c.take(p * oz2::packed_ld(q, 1)));
  w.scale = static_cast<float*>(c.take(sizeof(float) * p));
  if (oz2::few_rows(w.plan)) return w;  // takes any rows
  if (pack_v) w.v = static_cast<int8_t*>(c.take(r * oz2::packed_ld(q, 1)));
  w.partial = c.take(oz2::partial_bytes(w.plan, p, r));
  return w;
}

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

int status(hipError_t e) { return e == hipSuccess ? OZ2_OK : OZ2_ERR_HIP; }

}  // namespace

extern "C" {

int ozaki2_linear(int type, int p, int q, int r, const void* X, int ldx, const void* W, int ldw, const void* bias,
                  int act, const oz2_dropout_t* dropout, const void* R, int ldr, void* Z, int ldz, void* Y, int ldy,
                  void* work, size_t work_bytes, void* stream) {
  if (type != OZ2_BF16 && type != OZ2_F16) return OZ2_ERR_ARG;
  if (act < OZ2_ACT_NONE || act > OZ2_ACT_SILU || !drop_ok(dropout) || !sizes_ok(p, q, r)) return OZ2_ERR_ARG;
  const size_t e = elem_of(type);
  const Mat x{X, p, q, ldx, e}, w{W, r, q, ldw, e}, b{bias, 1, r, r, e}, res{R, p, r, ldr, e}, z{Z, p, r, ldz, e},
      y{Y, p, r, ldy, e};
  if (!ld_ok(x) || !ld_ok(w) || !ld_ok(res) || !ld_ok(z) || !ld_ok(y)) return OZ2_ERR_ARG;
  if (p == 0 || r == 0) return OZ2_OK;
  if (Y == nullptr || (q > 0 && (X == nullptr || W == nullptr))) return OZ2_ERR_ARG;
  if (!grid_ok(p, r)) return OZ2_ERR_UNSUPPORTED;
  if (overlap(y, x) || overlap(y, w) || overlap(y, b) || overlap(y, z) || (overlap(y, res) && !same(y, res))) return OZ2_ERR_ARG;
  if (overlap(z, x) || overlap(z, w) || overlap(z, b) || overlap(z, res)) return OZ2_ERR_ARG;
  const bool pack_x = !oz2::rows_aligned(X, ldx, q, 2), pack_w = !oz2::rows_aligned(W, ldw, q, 2);
  FwdWork ws;
  int rc = workspace(work, work_bytes, ws, [&](Carver& c) { return carve_fwd(c, p, q, r, pack_x, pack_w); });
  if (rc != OZ2_OK) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const long lp = oz2::packed_ld(q, 2);
  const oz2::PackJob jx{p, q, X, ldx, ws.x, lp}, jw{r, q, W, ldw, ws.w, lp};
  rc = status(oz2::launch_pack_rows(2, ws.x != nullptr ? &jx : nullptr, ws.w != nullptr ? &jw : nullptr, st));
  if (rc != OZ2_OK) return rc;
  // (where q is cut inside 16 bytes, both are packed, with zeros behind)
  oz2::Product pr{type,  false, p, r, q, ws.x != nullptr ? ws.x : X, ws.x != nullptr ? lp : ldx,
                  false, ws.w != nullptr ? ws.w : W, ws.w != nullptr ? lp : ldw, false, {}, ws.plan, ws.partial, false};
  pr.epi.bias = bias;
  pr.epi.act = act;
  pr.epi.drop = make_drop(dropout);
  pr.epi.res = R;
  pr.epi.ldr = ldr;
  pr.epi.z = Z;
  pr.epi.ldz = ldz;
  pr.epi.y = Y;
  pr.epi.ldy = ldy;
  return status(oz2::launch_product(pr, st));
}

int ozaki2_linear_bwd(int type, int p, int q, int r, const void* dY, int lddy, const void* X, int ldx, const void* W,
                      int ldw, const void* Z, int ldz, int act, const oz2_dropout_t* dropout, void* dX, int lddx,
                      void* dW, int lddw, void* dbias, void* work, size_t work_bytes, void* stream) {
  if (type != OZ2_BF16 && type != OZ2_F16) return OZ2_ERR_ARG;
  if (act < OZ2_ACT_NONE || act > OZ2_ACT_SILU || !drop_ok(dropout) || !sizes_ok(p, q, r)) return OZ2_ERR_ARG;
  const size_t e = elem_of(type);
  const Mat dy{dY, p, r, lddy, e}, x{X, p, q, ldx, e}, w{W, r, q, ldw, e}, z{Z, p, r, ldz, e}, dx{dX, p, q, lddx, e},
      dw{dW, r, q, lddw, e}, db{dbias, 1, r, r, e};
  if (!ld_ok(dy) || !ld_ok(x) || !ld_ok(w) || !ld_ok(z) || !ld_ok(dx) || !ld_ok(dw)) return OZ2_ERR_ARG;
  const bool want_dx = dX != nullptr && p > 0 && q > 0, want_dw = dW != nullptr && r > 0 && q > 0;
  const bool want_db = dbias != nullptr && r > 0;
  if (!want_dx && !want_dw && !want_db) return OZ2_OK;
  if (p > 0 && r > 0) {
    if (dY == nullptr || (act != OZ2_ACT_NONE && Z == nullptr)) return OZ2_ERR_ARG;
    if ((want_dx && W == nullptr) || (want_dw && X == nullptr)) return OZ2_ERR_ARG;
  }
  if ((want_dx && !grid_ok(p, q)) || (want_dw && !grid_ok(r, q))) return OZ2_ERR_UNSUPPORTED;
  const Mat* const outs[] = {&dx, &dw, &db};
  const Mat* const ins[] = {&dy, &x, &w, &z};
  for (const Mat* o : outs) {
    for (const Mat* i : ins)
      if (overlap(*o, *i)) return OZ2_ERR_ARG;
    for (const Mat* o2 : outs)
      if (o != o2 && overlap(*o, *o2)) return OZ2_ERR_ARG;
  }
  const oz2::Drop drop = make_drop(dropout);
  // dZ is dY itself without activation and dropout, if its rows are aligned; making it packs it.
  // Dropout's scale multiplies the products' sums, not dZ.
  const bool product = want_dx || want_dw;
  const bool make_dz = product && p > 0 && r > 0 && (act != OZ2_ACT_NONE || drop.t != 0 || !oz2::rows_aligned(dY, lddy, r, 2));
  const bool pack_x = want_dw && p > 0 && !oz2::rows_aligned(X, ldx, q, 2);
  const bool pack_w = want_dx && r > 0 && !oz2::rows_aligned(W, ldw, q, 2);
  BwdWork ws;
  int rc = workspace(work, work_bytes, ws,
                     [&](Carver& c) { return carve_bwd(c, p, q, r, want_dx && want_dw, make_dz, pack_x, pack_w); });
  if (rc != OZ2_OK) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const long lq = oz2::packed_ld(q, 2), lr = oz2::packed_ld(r, 2);
  if (make_dz || want_db) {
    rc = status(oz2::launch_grad_rows(type, p, r, dY, lddy, Z, ldz, act, drop, make_dz ? ws.dz : nullptr, lr,
                                      want_db ? ws.sums : nullptr, st));
    if (rc != OZ2_OK) return rc;
  }
  const oz2::PackJob jx{p, q, X, ldx, ws.x, lq}, jw{r, q, W, ldw, ws.w, lq};
  rc = status(oz2::launch_pack_rows(2, pack_x ? &jx : nullptr, pack_w ? &jw : nullptr, st));
  if (rc != OZ2_OK) return rc;
  const void* const dz = make_dz ? ws.dz : dY;
  const long lddz = make_dz ? lr : lddy;
  oz2::Product px{type, false, p, q, r, dz, lddz, false, pack_w ? ws.w : W, pack_w ? lq : ldw, true, {}, ws.dx, ws.partial_x, false};
  px.epi.y = dX;
  px.epi.ldy = lddx;
  px.epi.drop.scale = make_dz ? drop.scale / oz2::dz_factor(type == OZ2_F16, act) : 1.0f;
  oz2::Product pw{type, false, r, q, p, dz, lddz, true, pack_x ? ws.x : X, pack_x ? lq : ldx, true, {}, ws.dw, ws.partial_w, false};
  pw.epi.y = dW;
  pw.epi.ldy = lddw;
  pw.epi.drop.scale = px.epi.drop.scale;
  const oz2::ColumnSums sums{p > 0 ? oz2::grad_row_blocks(p, r) : 0, r, ws.sums, drop.scale, want_db ? dbias : nullptr};
  if (ws.paired) return status(oz2::launch_product_pair(type, px, pw, sums, st));
  if (want_db && (rc = status(oz2::launch_column_sums(type, sums, st))) != OZ2_OK) return rc;
  if (want_dx && (rc = status(oz2::launch_product(px, st))) != OZ2_OK) return rc;
  return want_dw ? status(oz2::launch_product(pw, st)) : OZ2_OK;
}

int ozaki2_dropout_add(int type, int p, int r, const void* X, int ldx, const void* R, int ldr,
                       const oz2_dropout_t* dropout, void* Y, int ldy, void* stream) {
  if (type < OZ2_BF16 || type > OZ2_F32 || !drop_ok(dropout) || !sizes_ok(p, 0, r)) return OZ2_ERR_ARG;
  const size_t e = elem_of(type);
  const Mat x{X, p, r, ldx, e}, res{R, p, r, ldr, e}, y{Y, p, r, ldy, e};
  if (!ld_ok(x) || !ld_ok(res) || !ld_ok(y)) return OZ2_ERR_ARG;
  if (p == 0 || r == 0) return OZ2_OK;
  if (X == nullptr || Y == nullptr) return OZ2_ERR_ARG;
  if ((overlap(y, x) && !same(y, x)) || (overlap(y, res) && !same(y, res))) return OZ2_ERR_ARG;
  return status(oz2::launch_dropout_add(type, p, r, X, ldx, R, ldr, make_drop(dropout), Y, ldy,
                                        static_cast<hipStream_t>(stream)));
}

int ozaki2_quantize_rows(int type, int p, int q, const void* X, int ldx, int8_t* Q, int ldq, float* scale, void* stream) {
  if (type < OZ2_BF16 || type > OZ2_F32 || !sizes_ok(p, q, 0)) return OZ2_ERR_ARG;
  const Mat x{X, p, q, ldx, elem_of(type)}, out{Q, p, q, ldq, 1}, sc{scale, 1, p, p, sizeof(float)};
  if (!ld_ok(x) || !ld_ok(out)) return OZ2_ERR_ARG;
  if (p == 0) return OZ2_OK;
  if (scale == nullptr || (q > 0 && (X == nullptr || Q == nullptr))) return OZ2_ERR_ARG;
  if (overlap(out, x) || overlap(sc, x) || overlap(sc, out)) return OZ2_ERR_ARG;
  return status(oz2::launch_quantize_rows(type, p, q, X, ldx, Q, ldq, q, scale, static_cast<hipStream_t>(stream)));
}

int ozaki2_linear_i8(int type, int p, int q, int r, const void* X, int ldx, const int8_t* V, int ldv, const float* t,
                     const void* bias, int act, const void* R, int ldr, void* Y, int ldy, void* work,
                     size_t work_bytes, void* stream) {
  if (type != OZ2_BF16 && type != OZ2_F16) return OZ2_ERR_ARG;
  if (act < OZ2_ACT_NONE || act > OZ2_ACT_SILU || !sizes_ok(p, q, r)) return OZ2_ERR_ARG;
  const size_t e = elem_of(type);
  const Mat x{X, p, q, ldx, e}, v{V, r, q, ldv, 1}, sc{t, 1, r, r, sizeof(float)}, b{bias, 1, r, r, e},
      res{R, p, r, ldr, e}, y{Y, p, r, ldy, e};
  if (!ld_ok(x) || !ld_ok(v) || !ld_ok(res) || !ld_ok(y)) return OZ2_ERR_ARG;
  if (p == 0 || r == 0) return OZ2_OK;
  if (q > OZ2_LINEAR_I8_MAX_Q || !grid_ok(p, r)) return OZ2_ERR_UNSUPPORTED;
  if (Y == nullptr || t == nullptr || (q > 0 && (X == nullptr || V == nullptr))) return OZ2_ERR_ARG;
  if (overlap(y, x) || overlap(y, v) || overlap(y, sc) || overlap(y, b) || (overlap(y, res) && !same(y, res))) return OZ2_ERR_ARG;
  const bool pack_v = !oz2::rows_aligned(V, ldv, q, 1);
  I8Work ws;
  int rc = workspace(work, work_bytes, ws, [&](Carver& c) { return carve_i8(c, p, q, r, pack_v); });
  if (rc != OZ2_OK) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const long lq = oz2::packed_ld(q, 1);
  const bool quantize = ws.q == nullptr;  // in the product
  if (!quantize) {
    rc = status(oz2::launch_quantize_rows(type, p, q, X, ldx, ws.q, lq, static_cast<int>(lq), ws.scale, st));
    if (rc != OZ2_OK) return rc;
  }
  const oz2::PackJob jv{r, q, V, ldv, ws.v, lq};
  if ((rc = status(oz2::launch_pack_rows(1, ws.v != nullptr ? &jv : nullptr, nullptr, st))) != OZ2_OK) return rc;
  // (where q is cut inside 16 bytes, V is packed too, or read element by element)
  oz2::Product pr{type,  true, p, r, q, quantize ? X : ws.q, quantize ? ldx : lq,
                  false, ws.v != nullptr ? ws.v : V, ws.v != nullptr ? lq : ldv, false, {}, ws.plan, ws.partial, quantize};
  pr.epi.bias = bias;
  pr.epi.act = act;
  pr.epi.res = R;
  pr.epi.ldr = ldr;
  pr.epi.y = Y;
  pr.epi.ldy = ldy;
  pr.epi.xs = ws.scale;
  pr.epi.ws = t;
  return status(oz2::launch_product(pr, st));
}

size_t ozaki2_linear_workspace_size(int call, int type, int p, int q, int r) {
  if ((type != OZ2_BF16 && type != OZ2_F16) || !sizes_ok(p, q, r)) return 0;
  Carver c;
  const bool aligned = (call & OZ2_LINEAR_ALIGNED) != 0;
  switch (call & ~OZ2_LINEAR_ALIGNED) {
    case OZ2_LINEAR_FWD:
      carve_fwd(c, p, q, r, !aligned, !aligned);
      break;
    case OZ2_LINEAR_BWD:
      {
        // with or without both products in one launch, the larger
        Carver both;
        carve_bwd(both, p, q, r, true, true, !aligned, !aligned);
        carve_bwd(c, p, q, r, false, true, !aligned, !aligned);
        c.used = std::max(c.used, both.used);
      }
      break;
    case OZ2_LINEAR_I8:
      carve_i8(c, p, q, r, !aligned);
      break;
  }
  return c.used;
}

}  // extern "C"
