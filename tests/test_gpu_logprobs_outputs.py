"""Every number the C entry point of tokens' log probabilities gives, each in a place of its own, against
their 64-bit forms, for rows of one workgroup and of several."""
import pytest

from tests import linear_reference as lin
from tests import logprobs_reference as ref
from tests.test_gpu_linear import BF16, F16, F32, oz, torch  # noqa: F401
from tests.test_gpu_linear_bounds import Place, Scratch, randn, stream
from tests.test_gpu_model_bounds import NAN, kind

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p, v", [(1, 1), (3, 13), (2, 4097), (9, 50003), (203, 9001), (1030, 777)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 5])
def test_outputs(oz, p, v, dtype, pad):  # noqa: F811
    top = min(v, 20)
    logits = Place(p, v, dtype, pad, NAN, randn(p, v, 1, 3.0))
    tokens = Place(1, p, torch.int64, 0, -9, torch.randint(0, v, (1, p), device="cuda"))
    lp, lse, h = (Place(1, p, F32, 0, 7.0) for _ in range(3))
    which, best = Place(1, p * top, torch.int64, 0, 7), Place(1, p * top, F32, 0, 7.0)
    work = Scratch(oz.ozaki2_token_logprobs_workspace_size(p, v, top))
    rc = oz.ozaki2_token_logprobs(kind(oz, dtype), p, v, logits.ptr, logits.ld, tokens.ptr, top, lp.ptr, lse.ptr, h.ptr, which.ptr,
                                  best.ptr, work.ptr, work.size, stream())
    assert rc == oz.OZ2_OK
    r, order = ref.rows(logits.view), ref.largest(logits.view, top)
    lin.assert_within(lp.view[0], *ref.given(r, tokens.view[0]), "logprob")
    lin.assert_within(lse.view[0], r.lse, r.err + 2 * ref.U * r.lse.abs(), "lse")
    lin.assert_within(h.view[0], r.entropy, r.err_h + 2 * ref.U * r.entropy, "entropy")
    assert torch.equal(which.view.view(p, top), order)
    lin.assert_within(best.view.view(p, top), *ref.top_values(r, order), "top_logprob")
    for name, t in dict(logits=logits, tokens=tokens, lp=lp, lse=lse, h=h, which=which, best=best).items():
        t.check(name)
    work.check()
