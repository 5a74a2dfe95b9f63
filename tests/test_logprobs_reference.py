"""The 64-bit gradient of log probabilities and entropy against differences (CPU)."""
import math

import pytest
import torch

from tests import logprobs_reference as ref


@pytest.mark.parametrize("parts", ["both", "logprob", "entropy"])
def test_gradient_against_differences(parts):
    g = torch.Generator().manual_seed(4)
    l = torch.randn(6, 9, generator=g, dtype=torch.float64) * 2
    l[1, 2:5] = -math.inf
    tokens = torch.tensor([0, 8, 3, -1, 4, 1])
    dlp = torch.randn(6, generator=g, dtype=torch.float64) if parts != "entropy" else None
    dh = torch.randn(6, generator=g, dtype=torch.float64) if parts != "logprob" else None

    def loss(l):
        r = ref.rows(l)
        total = 0.0
        if dlp is not None:
            total = total + (ref.given(r, tokens)[0] * dlp).sum()
        return total if dh is None else total + (r.entropy * dh).sum()

    keep, ref.rounding = ref.rounding, lambda y, dt: 0.0
    try:
        grad = ref.backward(l, tokens, dlp, dh)[0]
    finally:
        ref.rounding = keep
    step = 1e-6
    for i in range(6):
        for j in range(9):
            if l[i, j] == -math.inf:
                assert grad[i, j] == 0
                continue
            up, down = l.clone(), l.clone()
            up[i, j] += step
            down[i, j] -= step
            assert abs((loss(up) - loss(down)) / (2 * step) - grad[i, j]) < 1e-8
