"""The logits' gradient where nothing reaches a row: a padded place (a negative token) whose entropy has
no gradient.  Its logits may be anything, as what a padded row holds is never looked at; one NaN of
it would reach all of the weights' gradient through the product before."""
import math

import pytest

from tests import logprobs_reference as ref
from tests import linear_reference as lin
from tests.test_gpu_linear import BF16, F16, F32, normal, oz, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p, v", [(4, 3), (7, 1000), (6, 50001), (1100, 515)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("in_place", [False, True])
def test_nothing_comes_of_padded_rows(oz, p, v, dtype, in_place):  # noqa: F811
    l = normal(p, v, dtype, 1, 3.0, pad=3).clone()
    tokens = torch.randint(0, v, (p,), generator=torch.Generator().manual_seed(2)).cuda()
    padded = torch.arange(p, device="cuda") % 2 == 1
    tokens[padded] = -100
    for k, junk in enumerate((math.nan, math.inf, -math.inf)):
        l[1::2, k % v::3] = junk
    l[1] = math.nan
    r = ref.rows(l)
    dlp, dh = torch.randn(p, device="cuda"), torch.randn(p, device="cuda")
    dlp[padded] = math.nan
    dh[padded] = 0
    for d in (None, dh):
        got = oz.token_logprobs(l, tokens, entropy=True)
        assert (got.logprobs[padded] == 0).all()
        place = l.clone() if in_place else l
        grad = oz.token_logprobs_backward(dlp, place, tokens, got.lse, dentropy=d, entropy=None if d is None else got.entropy,
                                          out=place if in_place else None)
        assert (grad[padded] == 0).all()
        want, bound = ref.backward(l[~padded], tokens[~padded], dlp[~padded], None if d is None else d[~padded])
        # (lse and the entropy are the forward call's own here, off by its error)
        prob = (r.d - r.logs[:, None])[~padded].exp()
        more = dlp[~padded].abs().double()[:, None] * prob * (2 * r.err[~padded][:, None])
        if d is not None:
            share = d[~padded].abs().double()[:, None] * prob
            more = more + share * ((r.entropy[~padded] + 30)[:, None] * 2 * r.err[~padded][:, None] + r.err_h[~padded][:, None])
        lin.assert_within(grad[~padded], want, bound + more, "dlogits")
    # without a gradient of log probabilities, rows whose entropy has none
    grad = oz.token_logprobs_backward(None, l, None, got.lse, dentropy=dh, entropy=got.entropy)
    assert (grad[padded] == 0).all() and torch.isfinite(grad).all()
