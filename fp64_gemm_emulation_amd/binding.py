"""ctypes binding of liboz2.so (the C ABI in include/oz2.h).

Argument marshalling only: every step of the computation runs in the HIP library.
The functions named like the C entry points take plain integers / device pointers;
``dgemm`` and ``dgemm_debug``, and ``linear``, ``linear_backward``, ``dropout_add``,
``quantize_rows`` and ``linear_i8``, are conveniences over torch tensors (PyTorch supplies
device memory and the current stream, nothing else).

Loading fails loudly if the library has not been built: there is no fallback.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "liboz2.so")

OZ2_FAST, OZ2_ACCU = 0, 1
OZ2_OK, OZ2_ERR_ARG, OZ2_ERR_UNSUPPORTED, OZ2_ERR_WORKSPACE, OZ2_ERR_HIP = 0, 1, 2, 3, 4
OZ2_MIN_S, OZ2_MAX_S, OZ2_MAX_Q, OZ2_MAX_Q_P_DUMP, OZ2_X_LIMBS = 2, 20, 524287, 131071, 5
OZ2_OP_N, OZ2_OP_T = 0, 1
OZ2_FLAG_NONFINITE = 1
OZ2_NOALLOC_SCRATCH_BYTES = 256 << 20
MODES = {"fast": OZ2_FAST, "accu": OZ2_ACCU}
OZ2_BF16, OZ2_F16, OZ2_F32 = 0, 1, 2
OZ2_ACT_NONE, OZ2_ACT_RELU, OZ2_ACT_GELU, OZ2_ACT_GELU_TANH, OZ2_ACT_SILU = 0, 1, 2, 3, 4
OZ2_LINEAR_FWD, OZ2_LINEAR_BWD, OZ2_LINEAR_I8, OZ2_LINEAR_ALIGNED = 0, 1, 2, 16
OZ2_LINEAR_I8_MAX_Q = 131072
ACTIVATIONS = {"none": OZ2_ACT_NONE, "relu": OZ2_ACT_RELU, "gelu": OZ2_ACT_GELU, "gelu_tanh": OZ2_ACT_GELU_TANH,
               "silu": OZ2_ACT_SILU}


class Oz2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {ozaki2_status_string(status)} (status {status})")
        self.status = status


class OZ2Dump(ctypes.Structure):
    """Mirror of oz2_dump_t: device pointers (0 = skip)."""

    _fields_ = [(name, ctypes.c_void_p) for name in
                ("d", "b", "Ap", "Bp", "At", "Bt", "P", "R", "X",
                 "e", "f", "Abar", "Bbar", "rho", "gamma")]


class OZ2Dropout(ctypes.Structure):
    """Mirror of oz2_dropout_t."""

    _fields_ = [("probability", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64)]


def _share_hip_runtime():
    """PyTorch's wheel brings its own HIP runtime.  Where it is not loaded yet (torch imported
    after this module), load it now, so that the library binds to it: with the system's copy the
    process would hold two, and the library's launches on torch's memory and streams fail."""
    spec = importlib.util.find_spec("torch")
    for folder in (spec.submodule_search_locations or ()) if spec is not None else ():
        runtime = os.path.join(folder, "lib", "libamdhip64.so")
        if os.path.exists(runtime):
            ctypes.CDLL(runtime)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it first (python -m fp64_gemm_emulation_amd.build)")
    _share_hip_runtime()
    lib = ctypes.CDLL(LIB_PATH)
    i, vp, sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    sig = {
        "ozaki2_dgemm": (i, [i, i, i, vp, i, vp, i, vp, i, i, i, vp]),
        "ozaki2_dgemm_noalloc": (i, [i, i, i, vp, i, vp, i, vp, i, i, i, vp]),
        "ozaki2_dgemm_ex": (i, [i, i, i, i, i, ctypes.c_double, vp, i, vp, i, ctypes.c_double, vp, i, i, i, vp]),
        "ozaki2_dgemm_debug": (i, [i, i, i, vp, i, vp, i, vp, i, i, i, vp, ctypes.POINTER(OZ2Dump)]),
        "ozaki2_workspace_size": (sz, [i, i, i, i, i]),
        "ozaki2_set_workspace": (i, [vp, sz]),
        "ozaki2_release": (i, []),
        "ozaki2_timing_begin": (i, [i]),
        "ozaki2_timing_end": (i, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i)]),
        "ozaki2_get_stage_ms": (i, [ctypes.POINTER(ctypes.c_float)]),
        "ozaki2_get_flags": (i, [ctypes.POINTER(ctypes.c_uint)]),
        "ozaki2_moduli": (i, [i, ctypes.POINTER(i)]),
        "ozaki2_tau": (i, [i]),
        "ozaki2_status_string": (ctypes.c_char_p, [i]),
        "ozaki2_linear": (i, [i, i, i, i, vp, i, vp, i, vp, i, vp, vp, i, vp, i, vp, i, vp, sz, vp]),
        "ozaki2_linear_bwd": (i, [i, i, i, i, vp, i, vp, i, vp, i, vp, i, i, vp, vp, i, vp, i, vp, vp, sz, vp]),
        "ozaki2_dropout_add": (i, [i, i, i, vp, i, vp, i, vp, vp, i, vp]),
        "ozaki2_quantize_rows": (i, [i, i, i, vp, i, vp, i, vp, vp]),
        "ozaki2_linear_i8": (i, [i, i, i, i, vp, i, vp, i, vp, vp, i, vp, i, vp, i, vp, sz, vp]),
        "ozaki2_linear_workspace_size": (sz, [i, i, i, i, i]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_LIB = _load()


# --- entry points with the C names -------------------------------------------------
def ozaki2_dgemm(p, q, r, A, lda, B, ldb, C, ldc, s, mode, stream) -> int:
    return _LIB.ozaki2_dgemm(p, q, r, A, lda, B, ldb, C, ldc, s, mode, stream)


def ozaki2_dgemm_noalloc(p, q, r, A, lda, B, ldb, C, ldc, s, mode, stream) -> int:
    return _LIB.ozaki2_dgemm_noalloc(p, q, r, A, lda, B, ldb, C, ldc, s, mode, stream)


def ozaki2_dgemm_ex(transa, transb, p, q, r, alpha, A, lda, B, ldb, beta, C, ldc, s, mode, stream) -> int:
    return _LIB.ozaki2_dgemm_ex(transa, transb, p, q, r, alpha, A, lda, B, ldb, beta, C, ldc, s, mode, stream)


def ozaki2_dgemm_debug(p, q, r, A, lda, B, ldb, C, ldc, s, mode, stream, dump: OZ2Dump | None) -> int:
    return _LIB.ozaki2_dgemm_debug(p, q, r, A, lda, B, ldb, C, ldc, s, mode, stream,
                                   ctypes.byref(dump) if dump is not None else None)


def ozaki2_workspace_size(p, q, r, s, mode) -> int:
    return _LIB.ozaki2_workspace_size(p, q, r, s, mode)


def ozaki2_set_workspace(ptr, nbytes) -> int:
    return _LIB.ozaki2_set_workspace(ptr, nbytes)


def ozaki2_release() -> int:
    return _LIB.ozaki2_release()


def ozaki2_timing_begin(max_calls: int) -> int:
    return _LIB.ozaki2_timing_begin(max_calls)


def ozaki2_timing_end():
    """Returns (status, [scaling, residues, gemm, crt] ms summed, ncalls)."""
    ms = (ctypes.c_double * 4)()
    n = ctypes.c_int(0)
    rc = _LIB.ozaki2_timing_end(ms, ctypes.byref(n))
    return rc, list(ms), n.value


def ozaki2_get_stage_ms():
    """Returns (status, [scaling, residues, gemm, crt] ms of the most recent timed call)."""
    ms = (ctypes.c_float * 4)()
    rc = _LIB.ozaki2_get_stage_ms(ms)
    return rc, list(ms)


def ozaki2_get_flags():
    v = ctypes.c_uint(0)
    rc = _LIB.ozaki2_get_flags(ctypes.byref(v))
    return rc, v.value


def ozaki2_moduli(s: int):
    out = (ctypes.c_int * max(s, 1))()
    rc = _LIB.ozaki2_moduli(s, out)
    return rc, list(out)[:s]


def ozaki2_tau(s: int) -> int:
    return _LIB.ozaki2_tau(s)


def ozaki2_status_string(status: int) -> str:
    return _LIB.ozaki2_status_string(status).decode()


def _dropout_ref(dropout):
    return ctypes.addressof(dropout) if dropout is not None else None


def ozaki2_linear(type, p, q, r, X, ldx, W, ldw, bias, act, dropout: OZ2Dropout | None, R, ldr, Z, ldz, Y, ldy,
                  work, work_bytes, stream) -> int:
    return _LIB.ozaki2_linear(type, p, q, r, X, ldx, W, ldw, bias, act, _dropout_ref(dropout), R, ldr, Z, ldz, Y, ldy,
                              work, work_bytes, stream)


def ozaki2_linear_bwd(type, p, q, r, dY, lddy, X, ldx, W, ldw, Z, ldz, act, dropout: OZ2Dropout | None, dX, lddx,
                      dW, lddw, dbias, work, work_bytes, stream) -> int:
    return _LIB.ozaki2_linear_bwd(type, p, q, r, dY, lddy, X, ldx, W, ldw, Z, ldz, act, _dropout_ref(dropout), dX, lddx,
                                  dW, lddw, dbias, work, work_bytes, stream)


def ozaki2_dropout_add(type, p, r, X, ldx, R, ldr, dropout: OZ2Dropout | None, Y, ldy, stream) -> int:
    return _LIB.ozaki2_dropout_add(type, p, r, X, ldx, R, ldr, _dropout_ref(dropout), Y, ldy, stream)


def ozaki2_quantize_rows(type, p, q, X, ldx, Q, ldq, scale, stream) -> int:
    return _LIB.ozaki2_quantize_rows(type, p, q, X, ldx, Q, ldq, scale, stream)


def ozaki2_linear_i8(type, p, q, r, X, ldx, V, ldv, t, bias, act, R, ldr, Y, ldy, work, work_bytes, stream) -> int:
    return _LIB.ozaki2_linear_i8(type, p, q, r, X, ldx, V, ldv, t, bias, act, R, ldr, Y, ldy, work, work_bytes, stream)


def ozaki2_linear_workspace_size(call, type, p, q, r) -> int:
    return _LIB.ozaki2_linear_workspace_size(call, type, p, q, r)


# --- torch conveniences --------------------------------------------------------------
def _colmajor_ld(t, name):
    import torch
    if t.dtype != torch.float64 or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D float64 CUDA tensor")
    rows, cols = t.shape
    if rows == 0 or cols == 0:
        return max(1, rows)
    if t.stride(0) != 1 or (cols > 1 and t.stride(1) < rows):
        raise ValueError(f"{name} must be column-major (stride (1, ld >= rows)); use colmajor()")
    return t.stride(1) if cols > 1 else max(1, rows)


def colmajor(t):
    """Column-major copy of a 2-D tensor (same values, Fortran layout)."""
    return t.t().contiguous().t()


def empty_colmajor(rows, cols, device="cuda", dtype=None):
    import torch
    return torch.empty((cols, rows), dtype=dtype or torch.float64, device=device).t()


def _stream_ptr(stream, device):
    import torch
    st = stream if stream is not None else torch.cuda.current_stream(device)
    return st.cuda_stream


def _on_device(*tensors):
    """The operands' common device, made current for the call (the library works on the
    current device)."""
    import torch
    dev = tensors[0].device
    for t in tensors[1:]:
        if t is not None and t.device != dev:
            raise ValueError("all operands must be on the same device")
    return torch.cuda.device(dev)


def dgemm(A, B, s: int = 14, mode: str = "fast", out=None, stream=None):
    """C = A B (FP64, emulated) for column-major CUDA tensors; returns C (column-major)."""
    p, q = A.shape
    q2, r = B.shape
    if q != q2:
        raise ValueError("inner dimensions differ")
    C = out if out is not None else empty_colmajor(p, r, device=A.device)
    if tuple(C.shape) != (p, r):
        raise ValueError("out has the wrong shape")
    with _on_device(A, B, C):
        rc = ozaki2_dgemm(p, q, r, A.data_ptr(), _colmajor_ld(A, "A"), B.data_ptr(), _colmajor_ld(B, "B"),
                          C.data_ptr(), _colmajor_ld(C, "C"), s, MODES[mode], _stream_ptr(stream, A.device))
    if rc != OZ2_OK:
        raise Oz2Error(rc, "ozaki2_dgemm")
    return C


def dgemm_ex(A, B, transa: bool = False, transb: bool = False, alpha: float = 1.0, beta: float = 0.0,
             C=None, s: int = 14, mode: str = "fast", stream=None):
    """C = alpha op(A) op(B) + beta C for column-major CUDA tensors (op = transpose when
    transa / transb); C is created (and beta must be 0) when not given.  Returns C."""
    p, q = (A.shape[1], A.shape[0]) if transa else tuple(A.shape)
    q2, r = (B.shape[1], B.shape[0]) if transb else tuple(B.shape)
    if q != q2:
        raise ValueError("inner dimensions differ")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = empty_colmajor(p, r, device=A.device)
    if tuple(C.shape) != (p, r):
        raise ValueError("C has the wrong shape")
    with _on_device(A, B, C):
        rc = ozaki2_dgemm_ex(OZ2_OP_T if transa else OZ2_OP_N, OZ2_OP_T if transb else OZ2_OP_N, p, q, r,
                             float(alpha), A.data_ptr(), _colmajor_ld(A, "A"), B.data_ptr(), _colmajor_ld(B, "B"),
                             float(beta), C.data_ptr(), _colmajor_ld(C, "C"), s, MODES[mode],
                             _stream_ptr(stream, A.device))
    if rc != OZ2_OK:
        raise Oz2Error(rc, "ozaki2_dgemm_ex")
    return C


DUMP_FIELDS = ("d", "b", "Ap", "Bp", "At", "Bt", "P", "R", "X", "e", "f", "Abar", "Bbar", "rho", "gamma")


def dgemm_debug(A, B, s: int = 14, mode: str = "fast", want=DUMP_FIELDS, stream=None):
    """Run ozaki2_dgemm_debug; returns dict with C and the requested intermediates as
    device tensors in the layouts documented in include/oz2.h."""
    import torch
    p, q = A.shape
    _, r = B.shape
    dev = A.device
    C = empty_colmajor(p, r, device=dev)
    shapes = {
        "d": ((p,), torch.int32), "b": ((r,), torch.int32),
        "Ap": ((q, p), torch.float64), "Bp": ((r, q), torch.float64),   # column-major p x q / q x r
        "At": ((s, p, q), torch.int8), "Bt": ((s, r, q), torch.int8),
        "P": ((s, r, p), torch.int32), "R": ((s, r, p), torch.uint8),
        "X": ((r, p, OZ2_X_LIMBS), torch.int32),
        "e": ((p,), torch.int32), "f": ((r,), torch.int32),
        "Abar": ((p, q), torch.int8), "Bbar": ((r, q), torch.int8),
        "rho": ((p,), torch.int32), "gamma": ((r,), torch.int32),
    }
    bufs = {k: torch.zeros(*shapes[k][0], dtype=shapes[k][1], device=dev) for k in want}
    dump = OZ2Dump(**{k: (bufs[k].data_ptr() if bufs[k].numel() else None) for k in want})
    with _on_device(A, B, C):
        rc = ozaki2_dgemm_debug(p, q, r, A.data_ptr(), _colmajor_ld(A, "A"), B.data_ptr(), _colmajor_ld(B, "B"),
                                C.data_ptr(), _colmajor_ld(C, "C"), s, MODES[mode], _stream_ptr(stream, dev), dump)
    if rc != OZ2_OK:
        raise Oz2Error(rc, "ozaki2_dgemm_debug")
    if "Ap" in bufs:
        bufs["Ap"] = bufs["Ap"].t()
    if "Bp" in bufs:
        bufs["Bp"] = bufs["Bp"].t()
    bufs["C"] = C
    return bufs


# --- linear layers -------------------------------------------------------------------
# Row-major 2-D tensors, one token per row (a 3-D batch is passed as its reshape(-1, q)).
# Outputs and scratch are allocated on the stream of the call, so calls on different
# streams share nothing; operands made on another stream have to be ready on this one.
# With stream= given, the operands are recorded on it, so that their memory is not handed out
# again while the call reads it, and the outputs on the stream that was current, to which they
# return (waiting for the call there is the caller's part).
# A single token's layer takes a few microseconds on the GPU, so these functions look up
# attributes once, and torch itself on first use only.
_torch = None
_KINDS = {}          # torch dtype -> oz2_type_t
_raw_stream = None   # device index -> hipStream_t of its current stream
_current_device = None
_grad_enabled = None


def _use_torch():
    global _torch, _raw_stream, _current_device, _grad_enabled
    import torch
    _grad_enabled = torch.is_grad_enabled
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _KINDS.update({torch.bfloat16: OZ2_BF16, torch.float16: OZ2_F16, torch.float32: OZ2_F32})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)
    _torch = torch
    return torch


def _shape2(t, name):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a 2-D tensor, not {len(shape)}-D")
    return shape


def _kind(t, name, f32=False):
    code = _KINDS.get(t.dtype)
    if code is None or (code == OZ2_F32 and not f32):
        raise ValueError(f"{name} must be bfloat16 or float16" + (" or float32" if f32 else "") + f", not {t.dtype}")
    return code


def _check_operand(t, name, shape, dtype, dev):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if dev < 0 or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the device of the other operands")


def _rows(t, name, shape, dtype, dev):
    """(pointer, leading dimension) of a row-major matrix; (None, columns) for None."""
    rows, cols = shape
    if t is None:
        return None, cols or 1
    _check_operand(t, name, shape, dtype, dev)
    if rows == 0 or cols == 0:
        return t.data_ptr(), cols or 1
    ld, step = t.stride()
    if (step != 1 and cols > 1) or (ld < cols and rows > 1):
        raise ValueError(f"{name} must be row-major (stride (ld >= columns, 1)), not stride {tuple(t.stride())}")
    if rows == 1:
        ld = cols
    if ld >= 1 << 31:
        raise ValueError(f"{name}: the row stride does not fit 32 bits")
    return t.data_ptr(), ld


def _vector(t, name, n, dtype, dev):
    if t is None:
        return None
    _check_operand(t, name, (n,), dtype, dev)
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _activation(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, not {name!r}")
    return code


def _make_dropout(dropout, seed, offset):
    if dropout == 0.0:
        return None
    if not 0.0 <= dropout <= 1.0:
        raise ValueError("dropout must be a probability")
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("seed and offset must fit 64 bits")
    return OZ2Dropout(dropout, seed, offset)


def _no_autograd(name):
    """The functions here compute no gradient by themselves: an operand whose gradient autograd
    would be asked for is refused, rather than answered with a result that has lost it."""
    raise ValueError(f"{name} is not differentiated by autograd: call it under torch.no_grad() (or on detached tensors) "
                     "and take its gradients with linear_backward or dropout_add")


def _written(out):
    """`out` was written without torch's knowledge: autograd's check of saved tensors goes by
    its version."""
    if not out.is_inference():
        _torch.autograd.graph.increment_version(out)


class _NoContext:
    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_NO_CONTEXT = _NoContext()


class _OnStream:
    """The caller's stream made current, and what the call uses recorded on the streams that
    use it."""

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        self.before = _torch.cuda.current_stream(self.stream.device)
        self.context = _torch.cuda.stream(self.stream)
        self.context.__enter__()
        return self

    def __exit__(self, *exc):
        self.context.__exit__(*exc)

    def record(self, operands, outputs):
        for t in operands:
            if t is not None:
                t.record_stream(self.stream)
        for t in outputs:
            if t is not None:
                t.record_stream(self.before)


def _entered(dev, stream):
    """Context that makes the call's device and stream current while outputs and scratch are
    allocated and the library is entered (none where they are)."""
    if dev < 0:
        raise ValueError("operands must be CUDA tensors")
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("the stream belongs to another device than the operands")
        return _OnStream(stream)
    return _NO_CONTEXT if dev == _current_device() else _torch.cuda.device(dev)


def _aligned(row_bytes, *rows):
    """OZ2_LINEAR_ALIGNED if every (pointer, row stride in bytes) of rows of row_bytes is."""
    if row_bytes % 16:
        return 0
    for p, ld in rows:
        if p is not None and (p % 16 or ld % 16 or ld >= 1 << 24):
            return 0
    return OZ2_LINEAR_ALIGNED


def _scratch(call, kind, p, q, r, device):
    """(tensor, pointer, bytes) of the call's workspace."""
    n = _LIB.ozaki2_linear_workspace_size(call, kind, p, q, r)
    if n == 0:
        return None, None, 0
    t = _torch.empty(n, dtype=_torch.uint8, device=device)
    return t, t.data_ptr(), n


def linear(x, w, bias=None, activation: str = "none", residual=None, dropout: float = 0.0, seed: int = 0,
           offset: int = 0, return_z: bool = False, out=None, stream=None):
    """residual + D(act(x w^T + bias)) for x [p, q], w [r, q] in bfloat16 or float16, D the
    dropout of the C header; with return_z, (y, z), z the pre-activation for
    linear_backward.  `out` may be `residual` itself.  No autograd: operands that require a
    gradient are refused unless gradients are off."""
    torch = _torch or _use_torch()
    p, q = shape = _shape2(x, "x")
    r = _shape2(w, "w")[0]
    kind, act, drop = _kind(x, "x"), _activation(activation), _make_dropout(dropout, seed, offset)
    if _grad_enabled() and (x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad)
                            or (residual is not None and residual.requires_grad) or (out is not None and out.requires_grad)):
        _no_autograd("linear")
    dtype, dev, device = x.dtype, x.get_device(), x.device
    with _entered(dev, stream) as on:
        px, ldx = _rows(x, "x", shape, dtype, dev)
        pw, ldw = _rows(w, "w", (r, q), dtype, dev)
        pr, ldr = _rows(residual, "residual", (p, r), dtype, dev)
        pb = _vector(bias, "bias", r, dtype, dev)
        y = out if out is not None else x.new_empty((p, r))
        py, ldy = _rows(y, "out", (p, r), dtype, dev) if out is not None else (y.data_ptr(), r or 1)
        z = x.new_empty((p, r)) if return_z else None
        work, pwork, nwork = _scratch(OZ2_LINEAR_FWD | _aligned(2 * q, (px, 2 * ldx), (pw, 2 * ldw)), kind, p, q, r, device)
        rc = _LIB.ozaki2_linear(kind, p, q, r, px, ldx, pw, ldw, pb, act, _dropout_ref(drop), pr, ldr,
                                z.data_ptr() if return_z else None, r or 1, py, ldy, pwork, nwork, _raw_stream(dev))
        if on is not None:
            on.record((x, w, bias, residual, out), (y if out is None else None, z))
    if rc != OZ2_OK:
        raise Oz2Error(rc, "ozaki2_linear")
    if out is not None:
        _written(out)
    return (y, z) if return_z else y


def linear_backward(dy, x, w, z=None, activation: str = "none", dropout: float = 0.0, seed: int = 0, offset: int = 0,
                    needs=("x", "w", "bias"), stream=None):
    """(dx, dw, dbias) of linear from dy [p, r]; those not named in `needs` are None.  z is
    linear's pre-activation, needed unless activation is "none"; dropout, seed and offset have
    to be the forward call's.  The residual's gradient is dy itself."""
    torch = _torch or _use_torch()
    p, r = shape = _shape2(dy, "dy")
    q = _shape2(w, "w")[1]
    kind, act, drop = _kind(dy, "dy"), _activation(activation), _make_dropout(dropout, seed, offset)
    unknown = set(needs) - {"x", "w", "bias"}
    if unknown:
        raise ValueError(f"needs names {sorted(unknown)}: only x, w and bias have gradients here")
    if act != OZ2_ACT_NONE and z is None:
        raise ValueError("the gradient of an activation needs z")
    dtype, dev, device = dy.dtype, dy.get_device(), dy.device
    with _entered(dev, stream) as on:
        pdy, lddy = _rows(dy, "dy", shape, dtype, dev)
        px, ldx = _rows(x, "x", (p, q), dtype, dev)
        pw, ldw = _rows(w, "w", (r, q), dtype, dev)
        pz, ldz = _rows(z, "z", shape, dtype, dev)
        dx = dy.new_empty((p, q)) if "x" in needs else None
        dw = dy.new_empty((r, q)) if "w" in needs else None
        db = dy.new_empty((r,)) if "bias" in needs else None
        work, pwork, nwork = _scratch(OZ2_LINEAR_BWD | _aligned(2 * q, (px, 2 * ldx), (pw, 2 * ldw)), kind, p, q, r, device)
        rc = _LIB.ozaki2_linear_bwd(kind, p, q, r, pdy, lddy, px, ldx, pw, ldw, pz, ldz, act, _dropout_ref(drop),
                                    dx.data_ptr() if dx is not None else None, q or 1,
                                    dw.data_ptr() if dw is not None else None, q or 1,
                                    db.data_ptr() if db is not None else None, pwork, nwork, _raw_stream(dev))
        if on is not None:
            on.record((dy, x, w, z), (dx, dw, db))
    if rc != OZ2_OK:
        raise Oz2Error(rc, "ozaki2_linear_bwd")
    return dx, dw, db


def dropout_add(x, residual=None, dropout: float = 0.0, seed: int = 0, offset: int = 0, out=None, stream=None):
    """residual + D(x) for x [p, r] in bfloat16, float16 or float32; the gradient with respect
    to x is dropout_add(dy, None, ...) with the same dropout, seed and offset.  `out` may be x
    or residual itself.  No autograd, as linear."""
    torch = _torch or _use_torch()
    p, r = shape = _shape2(x, "x")
    kind, drop = _kind(x, "x", f32=True), _make_dropout(dropout, seed, offset)
    if _grad_enabled() and (x.requires_grad or (residual is not None and residual.requires_grad)
                            or (out is not None and out.requires_grad)):
        _no_autograd("dropout_add")
    dtype, dev = x.dtype, x.get_device()
    with _entered(dev, stream) as on:
        px, ldx = _rows(x, "x", shape, dtype, dev)
        pr, ldr = _rows(residual, "residual", shape, dtype, dev)
        y = out if out is not None else x.new_empty((p, r))
        py, ldy = _rows(y, "out", shape, dtype, dev) if out is not None else (y.data_ptr(), r or 1)
        rc = _LIB.ozaki2_dropout_add(kind, p, r, px, ldx, pr, ldr, _dropout_ref(drop), py, ldy, _raw_stream(dev))
        if on is not None:
            on.record((x, residual, out), (y if out is None else None,))
    if rc != OZ2_OK:
        raise Oz2Error(rc, "ozaki2_dropout_add")
    if out is not None:
        _written(out)
    return y


def quantize_rows(x, stream=None):
    """(int8 tensor, float32 scale of each row) of x [p, q] in bfloat16, float16 or float32."""
    torch = _torch or _use_torch()
    p, q = shape = _shape2(x, "x")
    kind = _kind(x, "x", f32=True)
    dev, device = x.get_device(), x.device
    with _entered(dev, stream) as on:
        px, ldx = _rows(x, "x", shape, x.dtype, dev)
        out = torch.empty((p, q), dtype=torch.int8, device=device)
        scale = torch.empty((p,), dtype=torch.float32, device=device)
        rc = _LIB.ozaki2_quantize_rows(kind, p, q, px, ldx, out.data_ptr(), q or 1, scale.data_ptr(), _raw_stream(dev))
        if on is not None:
            on.record((x,), (out, scale))
    if rc != OZ2_OK:
        raise Oz2Error(rc, "ozaki2_quantize_rows")
    return out, scale


def linear_i8(x, v, t, bias=None, activation: str = "none", residual=None, out=None, stream=None):
    """residual + act(x w^T + bias) with w held as (v, t) = quantize_rows(w): x [p, q] in
    bfloat16 or float16 is quantised by rows in the call.  `out` may be `residual` itself.  No
    autograd, as linear."""
    torch = _torch or _use_torch()
    p, q = shape = _shape2(x, "x")
    r = _shape2(v, "v")[0]
    kind, act = _kind(x, "x"), _activation(activation)
    if t is None:
        raise ValueError("t, the scales of v's rows, is needed")
    if _grad_enabled() and (x.requires_grad or t.requires_grad or (bias is not None and bias.requires_grad)
                            or (residual is not None and residual.requires_grad) or (out is not None and out.requires_grad)):
        _no_autograd("linear_i8")
    dtype, dev, device = x.dtype, x.get_device(), x.device
    with _entered(dev, stream) as on:
        px, ldx = _rows(x, "x", shape, dtype, dev)
        pv, ldv = _rows(v, "v", (r, q), torch.int8, dev)
        pt = _vector(t, "t", r, torch.float32, dev)
        pr, ldr = _rows(residual, "residual", (p, r), dtype, dev)
        pb = _vector(bias, "bias", r, dtype, dev)
        y = out if out is not None else x.new_empty((p, r))
        py, ldy = _rows(y, "out", (p, r), dtype, dev) if out is not None else (y.data_ptr(), r or 1)
        work, pwork, nwork = _scratch(OZ2_LINEAR_I8 | _aligned(q, (pv, ldv)), kind, p, q, r, device)
        rc = _LIB.ozaki2_linear_i8(kind, p, q, r, px, ldx, pv, ldv, pt, pb, act, pr, ldr, py, ldy, pwork, nwork,
                                   _raw_stream(dev))
        if on is not None:
            on.record((x, v, t, bias, residual, out), (y if out is None else None,))
    if rc != OZ2_OK:
        raise Oz2Error(rc, "ozaki2_linear_i8")
    if out is not None:
        _written(out)
    return y
