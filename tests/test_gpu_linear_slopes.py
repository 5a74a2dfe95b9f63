"""Slopes of the activations where the pre-activation is huge or no longer finite."""
import pytest

from tests import linear_reference as ref
from tests.test_gpu_linear import BF16, F16, oz, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ref.ACTS)
def test_slopes_of_huge_pre_activations(oz, act):  # noqa: F811
    """bfloat16's whole range, beyond where z * z and z's exponential leave f32's."""
    z = torch.tensor([1e4, 3e9, 1.8e19, 1.9e19, 1e20, 3e38], device="cuda")
    z = torch.cat([z, -z]).to(BF16)[None]
    n = z.shape[1]
    dy, w = torch.ones(1, n, dtype=BF16, device="cuda"), torch.ones(n, 8, dtype=BF16, device="cuda")
    dx, dw, db = oz.linear_backward(dy, torch.ones(1, 8, dtype=BF16, device="cuda"), w, z=z, activation=act)
    want = ref.slope(z.double(), act)[0]
    assert torch.equal(db.double(), want) and torch.equal(dw.double(), want[:, None].expand(n, 8))
    assert torch.equal(dx.double(), want.sum().expand(1, 8))


@pytest.mark.parametrize("act", ref.ACTS[1:])
def test_pre_activations_rounded_to_infinity(oz, act):  # noqa: F811
    """A pre-activation past f16's range is kept as an infinity although the layer's output is
    finite (it is taken of the unrounded sum): the slope there is its limit, 0 or 1, and the
    gradients of the row stay finite."""
    x = torch.full((3, 16), 300.0, dtype=F16, device="cuda")
    x[1] = 1.0
    w = torch.full((24, 16), 2.0 ** -6, dtype=F16, device="cuda")
    w[0], w[2] = -300.0, 300.0
    y, z = oz.linear(x, w, activation=act, return_z=True)
    assert torch.isinf(z[0, 0]) and z[0, 0] < 0 and y[0, 0] == 0 and torch.isinf(z[0, 2]) and torch.isfinite(z[1]).all()
    dy, x = torch.ones_like(y), x * 2.0 ** -8
    # (every slope has reached its limit well before 64)
    want, bound = ref.linear_backward(dy, x, w, z.clamp(-64, 64), act)
    for name, g, v, e in zip(("dx", "dw", "db"), oz.linear_backward(dy, x, w, z=z, activation=act), want, bound):
        ref.assert_within(g, v, e, name)
