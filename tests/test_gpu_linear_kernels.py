"""Every kernel of the linear-layer products at sizes that the library's own plan sends to it
(tests/linear_plans.py), in every type and layout, against the 64-bit forms."""
import pytest

from tests import linear_plans as plans
from tests import linear_reference as ref
from tests.test_gpu_linear import BF16, F16, normal, oz, run_linear, torch, vector  # noqa: F401

pytestmark = pytest.mark.gpu
TYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
# row strides: aligned for the copies, and not
PADS = pytest.mark.parametrize("pad", [0, 5])


@pytest.mark.parametrize("shape, tile, split", plans.FORWARD, ids=str)
@TYPES
@PADS
def test_linear(oz, shape, tile, split, dtype, pad):  # noqa: F811
    assert plans.kernel(plans.forward(*shape)) == (tile, split)
    p, q, r = shape
    print("linear", shape, tile, dtype, pad, flush=True)
    x, w = normal(p, q, dtype, 1, pad=pad), normal(r, q, dtype, 2, scale=q ** -0.5, pad=pad)
    b, res = vector(r, dtype, 3), normal(p, r, dtype, 4, pad=pad)
    y, z = run_linear(oz, x, w, "gelu", b, res, (0.1, 5, 6), True)
    wy, wz, ey, ez = ref.linear(x, w, b, "gelu", res, (0.1, 5, 6))
    ref.assert_within(y, wy, ey, "y")
    ref.assert_within(z, wz, ez, "z")
    plain = oz.linear(x, w)
    wy, _, ey, _ = ref.linear(x, w)
    ref.assert_within(plain, wy, ey, "no epilogue")


@pytest.mark.parametrize("shape, tile, split", plans.INT8, ids=str)
@TYPES
@PADS
def test_linear_i8(oz, shape, tile, split, dtype, pad):  # noqa: F811
    assert plans.kernel(plans.int8(*shape)) == (tile, split)
    p, q, r = shape
    print("linear_i8", shape, tile, dtype, pad, flush=True)
    x, w = normal(p, q, dtype, 1, pad=pad), normal(r, q, dtype, 2, scale=q ** -0.5)
    v, t = oz.quantize_rows(w)
    if pad:
        wide = torch.zeros(r, q + pad, dtype=torch.int8, device="cuda")
        wide[:, :q] = v
        v = wide[:, :q]
    b, res = vector(r, dtype, 3), normal(p, r, dtype, 4, pad=pad)
    want, bound = ref.linear_i8(x, v, t, b, "silu", res)
    ref.assert_within(oz.linear_i8(x, v, t, bias=b, activation="silu", residual=res), want, bound, "y")
    want, bound = ref.linear_i8(x, v, t)
    ref.assert_within(oz.linear_i8(x, v, t), want, bound, "no epilogue")


@pytest.mark.parametrize("shape, paired, dx, dw", plans.BACKWARD, ids=str)
@TYPES
@PADS
def test_linear_backward(oz, shape, paired, dx, dw, dtype, pad):  # noqa: F811
    got = plans.backward(*shape)
    assert (got[0], plans.kernel(got[1]), plans.kernel(got[2])) == (paired, dx, dw)
    p, q, r = shape
    for act, drop in (("none", None), ("gelu", (0.1, 9, 8))):
        print("linear_backward", shape, act, dtype, pad, flush=True)
        dy, x = normal(p, r, dtype, 1, pad=pad), normal(p, q, dtype, 2, pad=pad)
        w = normal(r, q, dtype, 3, scale=q ** -0.5, pad=pad)
        z = normal(p, r, dtype, 4, pad=pad) if act != "none" else None
        d = {} if drop is None else dict(dropout=drop[0], seed=drop[1], offset=drop[2])
        got = oz.linear_backward(dy, x, w, z=z, activation=act, **d)
        want, bound = ref.linear_backward(dy, x, w, z, act, drop)
        for name, g, v, e in zip(("dx", "dw", "db"), got, want, bound):
            ref.assert_within(g, v, e, f"{name} {act}")
