"""Gradients of the linear layer at the ends of the types' ranges, and how often they round."""
import pytest

from tests import linear_plans as plans
from tests import linear_reference as ref
from tests.test_gpu_linear import BF16, F16, normal, oz, torch  # noqa: F401

pytestmark = pytest.mark.gpu
TYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])

# both products in one launch, whole and split; apart, whole and split; rows that need packing
SHAPES = [(300, 200, 264), (256, 256, 1024), (478, 8, 8), (320, 2056, 4100), (203, 515, 3901), (3, 40, 56)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("prob", [0.0, 0.5, 0.9])
def test_large_f16_gradients_stay_finite(oz, shape, act, prob):  # noqa: F811
    """dY up to the largest f16, whose product with dropout's scale and a slope above one is
    beyond the type, with weights and inputs small enough for every gradient to be in range."""
    p, q, r = shape
    print("large f16", shape, act, prob, flush=True)
    drop = (prob, 3, 4)
    dy = normal(p, r, F16, 1)
    big = normal(p, r, F16, 2) > 1.5
    dy[big] = (65504.0 * torch.sign(dy[big].float())).half()
    z = normal(p, r, F16, 3, scale=1.5) if act != "none" else None
    x, w = normal(p, q, F16, 4, scale=2.0 ** -9 / p ** 0.5), normal(r, q, F16, 5, scale=2.0 ** -9 / r ** 0.5)
    dx, dw, _ = got = oz.linear_backward(dy, x, w, z=z, activation=act, dropout=prob, seed=3, offset=4)
    want, bound = ref.linear_backward(dy, x, w, z, act, drop if prob else None)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    for name, g, v, e in zip(("dx", "dw", "db"), got, want, bound):
        ref.assert_within(g, v, e, name)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act", ["none", "relu"])
@TYPES
def test_masked_gradients_round_once(oz, shape, act, dtype):  # noqa: F811
    """Where dZ is dY or nothing, times dropout's scale, the products' operands are exact: dX and
    dW are off by the sums' own rounding (32 bits) and one rounding to the type."""
    p, q, r = shape
    print("round once", shape, act, dtype, flush=True)
    drop = (0.1, 7, 8)
    dy, x, w = normal(p, r, dtype, 1), normal(p, q, dtype, 2), normal(r, q, dtype, 3, scale=q ** -0.5)
    z = normal(p, r, dtype, 4) if act == "relu" else None
    dx, dw, _ = oz.linear_backward(dy, x, w, z=z, activation=act, dropout=drop[0], seed=drop[1], offset=drop[2])
    (wx, ww, _), _ = ref.linear_backward(dy, x, w, z, act, drop)
    dz = ref.dropped(dy.double(), drop)[0] * (ref.slope(z.double(), act) if act == "relu" else 1.0)
    # the sums' bound of ref.linear_backward, the scale's multiplication in it
    ex = (r + 16) * 2.0 ** -23 * (dz.abs() @ w.double().abs())
    ew = (p + 16) * 2.0 ** -23 * (dz.abs().t() @ x.double().abs())
    ref.assert_within(dx, wx, ex * 1.01 + ref.rounding(wx, dtype), "dx")
    ref.assert_within(dw, ww, ew * 1.01 + ref.rounding(ww, dtype), "dw")


def test_shapes_reach_every_form():
    forms = {plans.backward(*s)[0] for s in SHAPES}
    split = {(plans.backward(*s)[0], plans.backward(*s)[k][1] > 1) for s in SHAPES for k in (1, 2)}
    assert forms == {False, True} and split == {(a, b) for a in (False, True) for b in (False, True)}
