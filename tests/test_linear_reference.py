"""The 64-bit forms that the GPU tests compare with, themselves checked on the CPU: the
generator against its published test vectors, activations' slopes and the layer's gradients
against differences."""
import numpy as np
import pytest
import torch

from tests import linear_reference as ref


@pytest.mark.parametrize("counter, key, want", [  # the vectors published with the generator
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_test_vectors(counter, key, want):
    assert tuple(ref.philox(counter, key)) == want


def test_draws_are_the_generators_lanes():
    rows, cols, seed, offset = 3, 19, 0x123456789ABCDEF0, (5 << 32) | 7
    u = ref.draws(rows, cols, seed, offset)
    for i in range(rows):
        for j in range(cols):
            n = i * 3 + j // 8
            words = ref.philox((n & 0xFFFFFFFF, n >> 32, 7, 5), (0x9ABCDEF0, 0x12345678))
            assert u[i, j] == words[j % 8 // 2] >> 16 * (j % 2) & 0xFFFF
    assert np.array_equal(ref.draws(1, cols, seed, offset, row0=2), u[2:])


def test_draws_are_uniform():
    u = ref.draws(512, 512, 99, 1) / 65536.0
    n = u.size
    # mean 1/2 and variance 1/12 within five standard errors
    assert abs(u.mean() - 0.5) < 5 * np.sqrt(1 / 12 / n)
    assert abs(u.var() - 1 / 12) < 5 * np.sqrt((1 / 80 - 1 / 144) / n)
    assert abs(np.corrcoef(u[:, :-1].ravel(), u[:, 1:].ravel())[0, 1]) < 5 / np.sqrt(n)


@pytest.mark.parametrize("act", ref.ACTS)
def test_slopes_against_differences(act):
    z = torch.linspace(-6, 6, 481, dtype=torch.float64) + 0.003
    h = 1e-6
    d = (ref.activate(z + h, act) - ref.activate(z - h, act)) / (2 * h)
    assert torch.allclose(ref.slope(z, act), d, atol=1e-8, rtol=0)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("drop", [None, (0.3, 11, 12)])
def test_gradients_against_differences(act, drop):
    g = torch.Generator().manual_seed(5)
    x, w, b, dy = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((7, 9), (11, 9), (11,), (7, 11)))

    def loss(x, w, b):
        return (ref.dropped(ref.activate(x @ w.t() + b, act), drop)[0] * dy).sum()

    dz, _ = ref.dropped(dy, drop)
    dz = dz * ref.slope(x @ w.t() + b, act)
    for k, grad in enumerate((dz @ w, dz.t() @ x, dz.sum(0))):
        step = torch.randn(*grad.shape, generator=g, dtype=torch.float64)
        h, args = 1e-6, [x, w, b]
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + h * step, args[k] - h * step
        assert abs((loss(*up) - loss(*down)) / (2 * h) - (grad * step).sum()) < 1e-6 * grad.norm() * step.norm()
