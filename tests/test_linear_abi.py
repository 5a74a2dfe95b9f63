"""The linear-layer entry points without a GPU: what they refuse, they refuse on the host
before anything is launched, and empty products return without a launch."""
import ctypes

import pytest
import torch

from fp64_gemm_emulation_amd import binding as oz

A, B, C, D, E, F = (0x10000000 * k for k in range(1, 7))  # never dereferenced
HUGE = (1 << 23) + 1
NAN = float("nan")


def call(fn, args, **kw):
    unknown = set(kw) - set(args)
    assert not unknown, unknown
    return fn(*{**args, **kw}.values())


LINEAR = dict(type=oz.OZ2_BF16, p=8, q=16, r=24, X=A, ldx=16, W=B, ldw=16, bias=C, act=oz.OZ2_ACT_GELU, dropout=None,
              R=D, ldr=24, Z=E, ldz=24, Y=F, ldy=24, work=None, work_bytes=0, stream=None)
BWD = dict(type=oz.OZ2_F16, p=8, q=16, r=24, dY=A, lddy=24, X=B, ldx=16, W=C, ldw=16, Z=D, ldz=24, act=oz.OZ2_ACT_SILU,
           dropout=None, dX=E, lddx=16, dW=F, lddw=16, dbias=F + 0x100000, work=None, work_bytes=0, stream=None)
DROP = dict(type=oz.OZ2_F32, p=8, r=24, X=A, ldx=24, R=B, ldr=24, dropout=None, Y=C, ldy=24, stream=None)
QUANT = dict(type=oz.OZ2_F32, p=8, q=16, X=A, ldx=16, Q=B, ldq=16, scale=C, stream=None)
I8 = dict(type=oz.OZ2_BF16, p=8, q=16, r=24, X=A, ldx=16, V=B, ldv=16, t=C, bias=D, act=oz.OZ2_ACT_RELU, R=E, ldr=24,
          Y=F, ldy=24, work=None, work_bytes=0, stream=None)
CALLS = {"linear": (oz.ozaki2_linear, LINEAR), "bwd": (oz.ozaki2_linear_bwd, BWD), "drop": (oz.ozaki2_dropout_add, DROP),
         "quant": (oz.ozaki2_quantize_rows, QUANT), "i8": (oz.ozaki2_linear_i8, I8)}


@pytest.mark.parametrize("name, kw", [
    ("linear", dict(type=oz.OZ2_F32)), ("linear", dict(type=-1)), ("linear", dict(act=5)), ("linear", dict(act=-1)),
    ("linear", dict(p=-1)), ("linear", dict(q=-1)), ("linear", dict(r=-1)), ("linear", dict(p=HUGE)),
    ("linear", dict(ldx=15)), ("linear", dict(ldw=15)), ("linear", dict(ldr=23)), ("linear", dict(ldz=23)),
    ("linear", dict(ldy=23)), ("linear", dict(X=None)), ("linear", dict(W=None)), ("linear", dict(Y=None)),
    ("linear", dict(dropout=oz.OZ2Dropout(-0.1, 0, 0))), ("linear", dict(dropout=oz.OZ2Dropout(1.1, 0, 0))),
    ("linear", dict(dropout=oz.OZ2Dropout(NAN, 0, 0))),
    ("linear", dict(Y=A)), ("linear", dict(Y=B + 2)), ("linear", dict(Y=C)), ("linear", dict(Y=E)),
    ("linear", dict(Y=D, ldy=25)), ("linear", dict(Y=D + 2)), ("linear", dict(Z=D)), ("linear", dict(Z=A)),
    ("bwd", dict(type=oz.OZ2_F32)), ("bwd", dict(act=9)), ("bwd", dict(Z=None)), ("bwd", dict(dY=None)),
    ("bwd", dict(X=None)), ("bwd", dict(W=None)), ("bwd", dict(lddy=23)), ("bwd", dict(ldz=23)), ("bwd", dict(lddx=15)),
    ("bwd", dict(lddw=15)), ("bwd", dict(dX=A)), ("bwd", dict(dW=E)), ("bwd", dict(dbias=D)),
    ("bwd", dict(dropout=oz.OZ2Dropout(2.0, 0, 0))), ("bwd", dict(work=0x101, work_bytes=1 << 30)),
    ("drop", dict(type=3)), ("drop", dict(p=-1)), ("drop", dict(X=None)), ("drop", dict(Y=None)), ("drop", dict(ldx=23)),
    ("drop", dict(ldr=23)), ("drop", dict(ldy=23)), ("drop", dict(Y=A + 4)), ("drop", dict(Y=B, ldy=32)),
    ("drop", dict(dropout=oz.OZ2Dropout(NAN, 0, 0))),
    ("quant", dict(type=-1)), ("quant", dict(q=-1)), ("quant", dict(X=None)), ("quant", dict(Q=None)),
    ("quant", dict(scale=None)), ("quant", dict(ldx=15)), ("quant", dict(ldq=15)), ("quant", dict(Q=A)),
    ("quant", dict(scale=B)),
    ("i8", dict(type=oz.OZ2_F32)), ("i8", dict(act=7)), ("i8", dict(X=None)), ("i8", dict(V=None)), ("i8", dict(t=None)),
    ("i8", dict(Y=None)), ("i8", dict(ldv=15)), ("i8", dict(Y=B)), ("i8", dict(Y=C)), ("i8", dict(Y=E, ldy=30)),
    ("i8", dict(work=0x101, work_bytes=1 << 30)),
])
def test_refused(name, kw):
    fn, args = CALLS[name]
    assert call(fn, args, **kw) == oz.OZ2_ERR_ARG


def test_unsupported_sizes():
    big = dict(p=1 << 23, r=1 << 20, ldr=1 << 20, ldz=1 << 20, ldy=1 << 20)  # more tiles than a grid holds
    assert call(oz.ozaki2_linear, LINEAR, **big, R=None, Z=None, Y=1 << 50, W=1 << 49) == oz.OZ2_ERR_UNSUPPORTED
    q = oz.OZ2_LINEAR_I8_MAX_Q + 1
    assert call(oz.ozaki2_linear_i8, I8, q=q, ldx=q, ldv=q) == oz.OZ2_ERR_UNSUPPORTED


def test_small_workspace_is_refused():
    need = oz.ozaki2_linear_workspace_size(oz.OZ2_LINEAR_BWD | oz.OZ2_LINEAR_ALIGNED, oz.OZ2_F16, 8, 16, 24)
    assert need > 0
    assert call(oz.ozaki2_linear_bwd, BWD, work=0x70000000, work_bytes=need - 1) == oz.OZ2_ERR_WORKSPACE
    need = oz.ozaki2_linear_workspace_size(oz.OZ2_LINEAR_I8 | oz.OZ2_LINEAR_ALIGNED, oz.OZ2_F16, 40, 16, 24)
    assert need > 0
    assert call(oz.ozaki2_linear_i8, I8, p=40, work=0x70000000, work_bytes=need - 1) == oz.OZ2_ERR_WORKSPACE
    assert oz.ozaki2_linear_workspace_size(oz.OZ2_LINEAR_BWD, oz.OZ2_F32, 8, 16, 24) == 0
    assert oz.ozaki2_linear_workspace_size(oz.OZ2_LINEAR_I8, oz.OZ2_F16, -8, 16, 24) == 0
    # a set workspace serves the call beyond its first 256 bytes
    assert oz.ozaki2_set_workspace(0x70000000, need) == oz.OZ2_OK
    try:
        assert call(oz.ozaki2_linear_i8, I8, p=40) == oz.OZ2_ERR_WORKSPACE
    finally:
        assert oz.ozaki2_set_workspace(None, 0) == oz.OZ2_OK


def test_workspace_sizes_of_empty_products():
    for call in (oz.OZ2_LINEAR_FWD, oz.OZ2_LINEAR_BWD, oz.OZ2_LINEAR_I8):
        for sizes in ((0, 16, 24), (40, 0, 24), (40, 16, 0), (0, 0, 0)):
            for flag in (0, oz.OZ2_LINEAR_ALIGNED):
                assert oz.ozaki2_linear_workspace_size(call | flag, oz.OZ2_BF16, *sizes) >= 0


def test_empty_calls_launch_nothing():
    assert call(oz.ozaki2_linear, LINEAR, p=0) == oz.OZ2_OK
    assert call(oz.ozaki2_linear, LINEAR, r=0, Y=None) == oz.OZ2_OK
    assert call(oz.ozaki2_linear_bwd, BWD, dX=None, dW=None, dbias=None) == oz.OZ2_OK
    assert call(oz.ozaki2_linear_bwd, BWD, p=0, dW=None, dbias=None) == oz.OZ2_OK
    assert call(oz.ozaki2_dropout_add, DROP, p=0) == oz.OZ2_OK
    assert call(oz.ozaki2_quantize_rows, QUANT, p=0) == oz.OZ2_OK
    assert call(oz.ozaki2_linear_i8, I8, r=0) == oz.OZ2_OK


def test_dropout_struct_layout():
    assert ctypes.sizeof(oz.OZ2Dropout) == 24 and oz.OZ2Dropout.seed.offset == 8 and oz.OZ2Dropout.offset.offset == 16


def test_tensor_wrappers_refuse():
    """Shapes, types, strides and devices, before any library call (host tensors throughout)."""
    x, w = torch.zeros(4, 6, dtype=torch.bfloat16), torch.zeros(5, 6, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        oz.linear(x, w)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        oz.linear(x.float(), w.float())
    with pytest.raises(ValueError, match="2-D"):
        oz.linear(x[0], w)
    with pytest.raises(ValueError, match="activation"):
        oz.linear(x, w, activation="tanh")
    with pytest.raises(ValueError, match="probability"):
        oz.linear(x, w, dropout=1.5)
    with pytest.raises(ValueError, match="64 bits"):
        oz.linear(x, w, dropout=0.5, seed=-1)
    with pytest.raises(ValueError, match="needs z"):
        oz.linear_backward(torch.zeros(4, 5, dtype=torch.float16), x, w, activation="relu")
    with pytest.raises(ValueError, match="needs names"):
        oz.linear_backward(torch.zeros(4, 5, dtype=torch.float16), x, w, needs=("residual",))
    with pytest.raises(ValueError):
        oz.linear(x, torch.zeros(5, 7, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="float32"):
        oz.quantize_rows(x.double())
