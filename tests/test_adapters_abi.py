"""ozaki2_linear_adapters without a GPU: what it refuses, it refuses on the host before anything is
launched; sizes of its workspace; operands whose gradient would be lost."""
import pytest
import torch

from fp64_gemm_emulation_amd import binding as oz

X, W, A, B, I, S, BIAS, R, Y = (0x10000000 * k for k in range(1, 10))  # never dereferenced
CALL = dict(type=oz.OZ2_BF16, p=8, q=16, r=24, X=X, ldx=16, W=W, ldw=16, bias=BIAS, act=oz.OZ2_ACT_GELU, adapters=None, R=R,
            ldr=24, Y=Y, ldy=24, work=None, work_bytes=0, stream=None)
ADAPTERS = dict(count=3, rank=4, A=A, lda=16, stride_a=64, B=B, ldb=4, stride_b=96, index=I, scale=S)


def call(adapters=None, **kw):
    assert not set(kw) - set(CALL) and not set(adapters or {}) - set(ADAPTERS)
    return oz.ozaki2_linear_adapters(*{**CALL, "adapters": oz.OZ2Adapters(**{**ADAPTERS, **(adapters or {})}), **kw}.values())


@pytest.mark.parametrize("kw", [
    dict(type=oz.OZ2_F32), dict(act=5), dict(p=-1), dict(q=-1), dict(r=-1), dict(ldx=15), dict(ldw=15), dict(ldr=23), dict(ldy=23),
    dict(X=None), dict(W=None), dict(Y=None), dict(Y=X), dict(Y=W), dict(Y=BIAS), dict(Y=R, ldy=25), dict(Y=A), dict(Y=A + 2 * 64),
    dict(Y=B + 2 * 180), dict(Y=I), dict(Y=S), dict(work=0x101, work_bytes=1 << 30), dict(adapters=None),
], ids=str)
def test_refused(kw):
    if "adapters" in kw:
        assert oz.ozaki2_linear_adapters(*CALL.values()) == oz.OZ2_ERR_ARG
    else:
        assert call(**kw) == oz.OZ2_ERR_ARG


@pytest.mark.parametrize("kw", [
    dict(count=-1), dict(rank=-1), dict(count=(1 << 23) + 1), dict(A=None), dict(B=None), dict(index=None), dict(lda=15), dict(ldb=3),
    dict(stride_a=-1), dict(stride_b=-1), dict(lda=1 << 40), dict(stride_b=1 << 40),
], ids=str)
def test_refused_adapters(kw):
    assert call(kw) == oz.OZ2_ERR_ARG


def test_other_statuses():
    assert call(dict(rank=257, ldb=257)) == oz.OZ2_ERR_UNSUPPORTED
    assert call(p=0) == oz.OZ2_OK and call(r=0, ldr=1, ldy=1) == oz.OZ2_OK
    assert call(work=0x100, work_bytes=64) == oz.OZ2_ERR_WORKSPACE
    size = oz.ozaki2_linear_adapters_workspace_size
    assert size(oz.OZ2_F32, 8, 16, 24, 3, 4, 0) == 0 and size(oz.OZ2_F16, 8, 16, 24, 3, 257, 0) == 0
    assert size(oz.OZ2_F16, 8, 16, 24, 3, -1, 0) == 0 and size(oz.OZ2_F16, 8, 16, 24, -1, 4, 0) == 0
    for p, q, r in ((1, 2048, 8192), (37, 8192, 2048), (8192, 2048, 8192), (777, 1999, 4099)):
        base = oz.ozaki2_linear_workspace_size(oz.OZ2_LINEAR_FWD, oz.OZ2_F16, p, q, r)
        assert size(oz.OZ2_F16, p, q, r, 3, 0, 0) == base and size(oz.OZ2_F16, p, q, r, 0, 50, 0) == base
        assert base + 4 * p * 64 <= size(oz.OZ2_F16, p, q, r, 3, 56, 0) <= base + (16 * 4 + 2) * p * 64 + 512
        packed = 2 * 3 * r * 56 if p > 16 else 0
        assert size(oz.OZ2_F16, p, q, r, 3, 50, 0) >= size(oz.OZ2_F16, p, q, r, 3, 56, 0) + packed


SIZES = dict(x=(4, 16), w=(8, 16), a=(3, 2, 16), b=(3, 8, 2), scale=(3,), bias=(8,), residual=(4, 8), out=(4, 8))


def make(grad=None):
    t = {k: torch.zeros(s, dtype=torch.float32 if k == "scale" else torch.float16).requires_grad_(k == grad) for k, s in SIZES.items()}
    return dict(t, index=torch.zeros(4, dtype=torch.int32))


@pytest.mark.parametrize("operand", list(SIZES))
def test_a_lost_gradient_is_refused(operand):
    with pytest.raises(ValueError, match="autograd"):
        oz.linear_adapters(**make(operand))
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        oz.linear_adapters(**make(operand))


def test_refused_by_the_binding():
    with pytest.raises(ValueError, match="index"):
        oz.linear_adapters(**dict(make(), index=None))
    with pytest.raises(ValueError, match="3-D"):
        oz.linear_adapters(**dict(make(), a=torch.zeros(2, 16).half()))
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        oz.linear_adapters(**dict(make(), x=torch.zeros(4, 16)))
