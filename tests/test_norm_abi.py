"""The norm's entry points without a GPU: what they refuse, they refuse on the host before
anything is launched; empty sizes return without a launch; operands whose gradient would be lost
are refused."""
import pytest
import torch

from fp64_gemm_emulation_amd import binding as oz

A, B, C, D, E, F = (0x10000000 * k for k in range(1, 7))  # never dereferenced
NAN = float("nan")
NORM = dict(type=oz.OZ2_BF16, p=8, q=16, X=A, ldx=16, R=B, ldr=16, w=C, eps=1e-6, H=D, ldh=16, Y=E, ldy=16, stream=None)
I8 = dict(type=oz.OZ2_F16, p=8, q=16, X=A, ldx=16, R=B, ldr=16, w=C, eps=1e-6, H=D, ldh=16, Q=E, ldq=16, scale=F, stream=None)
BWD = dict(type=oz.OZ2_F32, p=8, q=16, dY=A, lddy=16, H=B, ldh=16, w=C, eps=1e-6, dH=D, lddh=16, dX=E, lddx=16, dw=F,
           work=None, work_bytes=0, stream=None)
ROWS = dict(type=oz.OZ2_BF16, p=8, q=16, r=24, Q=A, ldq=16, s=A + 0x100000, V=B, ldv=16, t=C, bias=D, act=oz.OZ2_ACT_RELU,
            R=E, ldr=24, Y=F, ldy=24, work=None, work_bytes=0, stream=None)
CALLS = {"norm": (oz.ozaki2_rms_norm, NORM), "i8": (oz.ozaki2_rms_norm_i8, I8), "bwd": (oz.ozaki2_rms_norm_bwd, BWD),
         "rows": (oz.ozaki2_linear_i8_rows, ROWS)}


def call(name, **kw):
    fn, args = CALLS[name]
    assert not set(kw) - set(args)
    return fn(*{**args, **kw}.values())


@pytest.mark.parametrize("name, kw", [
    *((n, kw) for n in ("norm", "i8", "bwd") for kw in (
        dict(type=3), dict(type=-1), dict(p=-1), dict(q=-1), dict(p=(1 << 23) + 1), dict(eps=0.0), dict(eps=-1e-6), dict(eps=1e-39),
        dict(eps=NAN), dict(eps=float("inf")))),
    *((n, kw) for n in ("norm", "i8") for kw in (
        dict(X=None), dict(ldx=15), dict(ldr=15), dict(ldh=15), dict(H=A + 2), dict(H=B, ldh=24), dict(H=C))),
    ("norm", dict(Y=None)), ("norm", dict(ldy=15)), ("norm", dict(Y=D)), ("norm", dict(Y=C)), ("norm", dict(Y=A + 2)),
    ("norm", dict(Y=B, ldy=17)), ("norm", dict(H=A, Y=A)),
    ("i8", dict(Q=None)), ("i8", dict(scale=None)), ("i8", dict(ldq=15)), ("i8", dict(Q=A)), ("i8", dict(Q=B)),
    ("i8", dict(Q=D)), ("i8", dict(scale=E)), ("i8", dict(scale=C)), ("i8", dict(scale=A)),
    ("bwd", dict(dY=None)), ("bwd", dict(H=None)), ("bwd", dict(lddy=15)), ("bwd", dict(ldh=15)), ("bwd", dict(lddh=15)),
    ("bwd", dict(lddx=15)), ("bwd", dict(dX=B)), ("bwd", dict(dX=A + 4)), ("bwd", dict(dX=C)), ("bwd", dict(dw=E)),
    ("bwd", dict(dw=A)), ("bwd", dict(dw=C)), ("bwd", dict(work=0x101, work_bytes=1 << 30)),
    ("rows", dict(type=oz.OZ2_F32)), ("rows", dict(Q=None)), ("rows", dict(s=None)), ("rows", dict(t=None)),
    ("rows", dict(ldq=15)), ("rows", dict(Y=A)), ("rows", dict(Y=A + 0x100000)), ("rows", dict(Y=None)), ("rows", dict(act=7)),
])
def test_refused(name, kw):
    assert call(name, **kw) == oz.OZ2_ERR_ARG


def test_other_statuses():
    wide = oz.OZ2_NORM_MAX_Q + 1
    lds = {"norm": ("ldx", "ldr", "ldh", "ldy"), "i8": ("ldx", "ldr", "ldh", "ldq"), "bwd": ("lddy", "ldh", "lddh", "lddx")}
    for name, names in lds.items():
        assert call(name, p=1, q=wide, **dict.fromkeys(names, wide)) == oz.OZ2_ERR_UNSUPPORTED
        assert call(name, p=0, **({"dw": None} if name == "bwd" else {})) == oz.OZ2_OK
    assert call("norm", q=0) == oz.OZ2_OK and call("bwd", q=0) == oz.OZ2_OK
    assert call("bwd", dX=None, dw=None) == oz.OZ2_OK
    assert call("bwd", work=0x100, work_bytes=16) == oz.OZ2_ERR_WORKSPACE
    assert oz.ozaki2_rms_norm_bwd_workspace_size(3, 8, 16) == 0
    assert oz.ozaki2_rms_norm_bwd_workspace_size(oz.OZ2_F32, 8, wide) == 0
    assert oz.ozaki2_rms_norm_bwd_workspace_size(oz.OZ2_F32, 8, 16) >= 64
    assert call("rows", p=0, s=None) == oz.OZ2_OK


SIZES = dict(x=(4, 16), weight=(16,), residual=(4, 16), hidden=(4, 16))


@pytest.mark.parametrize("name, operand", [(n, o) for n in ("rms_norm", "rms_norm_i8") for o in (*SIZES, "out")
                                           if n == "rms_norm" or o != "out"])
def test_a_lost_gradient_is_refused(name, operand):
    sizes = dict(SIZES, out=(4, 16)) if name == "rms_norm" else SIZES
    make = lambda grad: {k: torch.zeros(s).requires_grad_(k == grad) for k, s in sizes.items()}  # noqa: E731
    with pytest.raises(ValueError, match="autograd"):
        getattr(oz, name)(**make(operand))
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        getattr(oz, name)(**make(operand))


def test_refused_by_the_binding():
    x, s = torch.zeros(4, 16), torch.zeros(4)
    with pytest.raises(ValueError, match="hidden"):
        oz.rms_norm(x, hidden=x)
    with pytest.raises(ValueError, match="needs"):
        oz.rms_norm_backward(x, x, needs=("w",))
    with pytest.raises(ValueError, match="2-D"):
        oz.rms_norm(torch.zeros(16))
    with pytest.raises(ValueError, match="float32"):
        oz.rms_norm(x.double())
    v, t = torch.zeros(8, 16, dtype=torch.int8), torch.zeros(8)
    with pytest.raises(ValueError, match="dtype"):
        oz.linear_i8(torch.zeros(4, 16, dtype=torch.int8), v, t, x_scale=s)
    with pytest.raises(ValueError, match="dtype"):
        oz.linear_i8(x.half(), v, t, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="autograd"):
        oz.linear_i8(torch.zeros(4, 16, dtype=torch.int8), v, t, x_scale=s.requires_grad_(), dtype=torch.float16)
