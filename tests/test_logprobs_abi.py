"""The entry points of tokens' log probabilities without a GPU: what they refuse, they refuse on the
host before anything is launched."""
import pytest
import torch

from fp64_gemm_emulation_amd import binding as oz

A, B, C, D, E, F, G, H = (0x10000000 * k for k in range(1, 9))  # never dereferenced
FWD = dict(type=oz.OZ2_BF16, p=8, v=100, L=A, ldl=100, tokens=B, top=5, logprob=C, lse=D, entropy=E, top_tokens=F,
           top_logprob=G, work=None, work_bytes=0, stream=None)
BWD = dict(type=oz.OZ2_F32, p=8, v=100, dlogprob=A, L=B, ldl=100, tokens=C, lse=D, dentropy=E, entropy=F, dL=G, lddl=100,
           stream=None)
CALLS = {"fwd": (oz.ozaki2_token_logprobs, FWD), "bwd": (oz.ozaki2_token_logprobs_bwd, BWD)}


def call(name, **kw):
    fn, args = CALLS[name]
    assert not set(kw) - set(args)
    return fn(*{**args, **kw}.values())


@pytest.mark.parametrize("name, kw", [
    *((n, kw) for n in CALLS for kw in (dict(type=3), dict(type=-1), dict(p=-1), dict(v=-1), dict(v=(1 << 23) + 1), dict(L=None),
                                        dict(ldl=99), dict(tokens=None))),
    ("fwd", dict(top=-1)), ("fwd", dict(top=65)), ("fwd", dict(v=4, ldl=4)), ("fwd", dict(top_tokens=None)),
    ("fwd", dict(top_logprob=None)), ("fwd", dict(lse=C)), ("fwd", dict(lse=C + 28)), ("fwd", dict(logprob=A)),
    ("fwd", dict(entropy=B)), ("fwd", dict(top_logprob=F)), ("fwd", dict(top_tokens=A + 200)),
    ("fwd", dict(work=0x101, work_bytes=1 << 30)),
    ("bwd", dict(lse=None)), ("bwd", dict(dL=None)), ("bwd", dict(entropy=None)), ("bwd", dict(lddl=99)), ("bwd", dict(dL=B + 4)),
    ("bwd", dict(dL=B, lddl=101)), ("bwd", dict(dL=A)), ("bwd", dict(dL=D)), ("bwd", dict(dL=E)), ("bwd", dict(dL=F)), ("bwd", dict(dL=C)),
])
def test_refused(name, kw):
    assert call(name, **kw) == oz.OZ2_ERR_ARG


def test_other_statuses():
    assert call("fwd", p=0) == oz.OZ2_OK
    assert call("bwd", p=0) == oz.OZ2_OK and call("bwd", v=0, ldl=1, lddl=1) == oz.OZ2_OK
    assert call("fwd", v=100000, ldl=100000, work=0x100, work_bytes=64) == oz.OZ2_ERR_WORKSPACE
    size = oz.ozaki2_token_logprobs_workspace_size
    assert size(8, 100, 5) == 0 and size(-1, 100, 0) == 0 and size(8, 100, 65) == 0
    assert size(1, 100000, 20) > size(1, 100000, 0) > 0 and size(5000, 100000, 20) == 0


def test_refused_by_the_binding():
    l, t = torch.zeros(4, 16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="autograd"):
        oz.token_logprobs(l.clone().requires_grad_(), t)
    for off in (torch.no_grad, torch.inference_mode):
        with off(), pytest.raises(ValueError, match="CUDA"):
            oz.token_logprobs(l.clone().requires_grad_(), t)
    for top in (-1, 17):
        with pytest.raises(ValueError, match="top"):
            oz.token_logprobs(l, t, top=top)
    with pytest.raises(ValueError, match="float32"):
        oz.token_logprobs(l.double(), t)
    s = torch.zeros(4)
    with pytest.raises(ValueError, match="tokens"):
        oz.token_logprobs_backward(s, l, None, s)
    with pytest.raises(ValueError, match="entropy"):
        oz.token_logprobs_backward(s, l, t, s, dentropy=s)
    with pytest.raises(ValueError, match="lse"):
        oz.token_logprobs_backward(s, l, t, None)
    with pytest.raises(ValueError, match="CUDA"):
        oz.token_logprobs_backward(s, l, t, s)
    with pytest.raises(ValueError, match="autograd"):
        oz.token_logprobs_backward(s, l, t, s, out=l.clone().requires_grad_())
