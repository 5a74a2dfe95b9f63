"""The norm's 64-bit gradient against differences of its 64-bit form (CPU)."""
import pytest
import torch

from tests import norm_reference as ref


@pytest.mark.parametrize("with_weight", [False, True])
@pytest.mark.parametrize("with_stream", [False, True])
def test_gradient_against_differences(with_weight, with_stream):
    g = torch.Generator().manual_seed(3)
    new = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    h, dy, dh, eps = new(5, 7), new(5, 7), new(5, 7) if with_stream else None, 1e-3
    w = new(7) if with_weight else None

    def loss(h, w):
        total = (ref.norm(h, w, eps)[0] * dy).sum()
        return total if dh is None else total + (h * dh).sum()

    # (64-bit inputs: the type is only used for the bounds' rounding)
    as_type = lambda t: None if t is None else t  # noqa: E731
    orig = ref.rounding
    ref.rounding = lambda y, dt: 0.0
    try:
        (dx, dw), _ = ref.backward(dy, h, as_type(w), dh, eps)
    finally:
        ref.rounding = orig
    step = 1e-5
    for t, grad in ((h, dx), (w, dw)) if with_weight else ((h, dx),):
        flat = t.view(-1)
        for i in range(flat.numel()):
            at = flat[i].item()
            flat[i] = at + step
            up = loss(h, w)
            flat[i] = at - step
            down = loss(h, w)
            flat[i] = at
            assert abs((up - down) / (2 * step) - grad.reshape(-1)[i]) < 1e-8
