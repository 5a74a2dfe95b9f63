"""Log probabilities of tokens on the GPU against their 64-bit forms (tests/logprobs_reference.py,
which derives the bounds): sizes, types and strides, masks that leave little or nothing, ties
and orders that the selection of the largest has to go through, values at the ends of the types'
ranges, in place, streams and graphs."""
import math

import pytest

from tests import linear_reference as lin
from tests import logprobs_reference as ref
from tests.test_gpu_linear import BF16, F16, F32, normal, oz, torch  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = {"bf16": BF16, "f16": F16, "f32": F32}
# one workgroup to a row and several, rows that end inside a chunk of eight, an unrolled step or a part
SHAPES = [(1, 1), (3, 2), (2, 7), (5, 65), (4, 1000), (2, 4096), (3, 4104), (1, 8191), (2, 8192), (17, 8200), (1, 32771), (7, 50001),
          (1, 131072), (1100, 1531), (1030, 9001)]


def tokens_of(p, v, seed):
    t = torch.randint(0, v, (p,), generator=torch.Generator().manual_seed(seed)).cuda()
    if p > 1:
        t[::7] = -1
    return t


def check(oz, l, tokens, top, entropy=True):  # noqa: F811
    got, r = oz.token_logprobs(l, tokens, top=top, entropy=entropy), ref.rows(l)
    lin.assert_within(got.lse, r.lse, r.err + 2 * ref.U * torch.nan_to_num(r.lse.abs(), posinf=0.0), "lse")
    if tokens is not None:
        lin.assert_within(got.logprobs, *ref.given(r, tokens), "logprobs")
    if entropy:
        lin.assert_within(got.entropy, r.entropy, r.err_h + 2 * ref.U * torch.nan_to_num(r.entropy), "entropy")
    if top:
        which = ref.largest(l, top)
        assert torch.equal(got.top_tokens, which)
        lin.assert_within(got.top_logprobs, *ref.top_values(r, which), "top_logprobs")
    return got


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("type", list(TYPES))
def test_logprobs(oz, shape, type):  # noqa: F811
    (p, v), dt = shape, TYPES[type]
    for k, (top, entropy, pad, shift) in enumerate([(20, True, 0, 0), (0, True, 3, 1), (1, False, 8, 0), (64, False, 5, 3), (0, False, 0, 0)]):
        print("logprobs", shape, type, top, entropy, pad, flush=True)
        l = normal(p, v, dt, k, 3.0, pad=pad, shift=shift)
        check(oz, l, tokens_of(p, v, k), min(top, v), entropy)
    got = oz.token_logprobs(l)
    assert got.logprobs is None and got.entropy is None and got.top_tokens is None and got.top_logprobs is None


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("type", list(TYPES))
def test_backward(oz, shape, type):  # noqa: F811
    (p, v), dt = shape, TYPES[type]
    g = torch.Generator().manual_seed(5)
    dlp, dh = torch.randn(p, generator=g).cuda(), torch.randn(p, generator=g).cuda()
    for k, (a, b, pad, shift) in enumerate([(dlp, dh, 0, 0), (dlp, None, 3, 1), (None, dh, 8, 0)]):
        print("backward", shape, type, k, flush=True)
        l, t = normal(p, v, dt, k, 3.0, pad=pad, shift=shift), tokens_of(p, v, k)
        r = ref.rows(l)
        kw = dict(dentropy=b, entropy=None if b is None else r.entropy.float())
        got = oz.token_logprobs_backward(a, l, t, r.lse.float(), **kw)
        lin.assert_within(got, *ref.backward(l, t, a, b), "dlogits")
        assert torch.equal(oz.token_logprobs_backward(a, l, t, r.lse.float(), out=l, **kw), got) and torch.equal(l, got)


@pytest.mark.parametrize("v", [1000, 9001, 70000])
@pytest.mark.parametrize("many", [False, True])
def test_orders(oz, v, many):  # noqa: F811
    """Rows that the selection of the largest does not meet in random order, alone (several
    workgroups to a row where it is long) and among so many rows that each has one."""
    g = torch.Generator(device="cuda").manual_seed(6)
    i = torch.arange(v, device="cuda")
    special = torch.stack([
        torch.zeros(v, device="cuda"), i * 0.25 % 977, -(i * 0.25 % 977), i / 64, -i / 64.0,
        torch.where(i // 8 % 256 < 63, 10.0, 0.0),            # all that is large in 63 threads' chunks
        torch.where(i // 8 % 256 < 64, 10.0 + i % 977 / 64, 0.0),
        torch.where(i // 8 % 256 < 64, 12.0 - i % 977 / 64, 0.0),
        (i % 3).float(), torch.where(i < v - 3, -math.inf, 1.0), torch.where(i == v // 2, 5.0, -math.inf),
        torch.where(i % 2 == 0, 0.0, -0.0), torch.randint(0, 4, (v,), generator=g, device="cuda").float(),
        torch.full((v,), -math.inf, device="cuda"),
    ])
    if many:
        special = special.repeat(-(-1040 // len(special)), 1) if v < 70000 else special.repeat(75, 1)
    t = tokens_of(len(special), v, 1)
    for dt in (F32, BF16):
        l = special.to(dt)
        for top in (1, 20, 64):
            print("orders", v, many, dt, top, flush=True)
            if many and top == 20:
                continue
            check(oz, l, t, top)


@pytest.mark.parametrize("v", [40, 9001])
def test_ends_of_the_range(oz, v):  # noqa: F811
    for dt in TYPES.values():
        low, high = torch.finfo(dt).min, torch.finfo(dt).max
        l = normal(12, v, dt, 3, 2.0).clone()
        l[0] = -math.inf
        l[1] = low
        l[2] = high
        l[3, 1:] = low
        l[4, ::2] = low
        l[5, ::2] = -math.inf
        l[6, v - 1] = math.nan
        l[7, v // 2] = math.inf
        l[8] = (l[8].float() * (100 if dt == F16 else 1e6)).to(dt)
        l[9, : v - 1] = -math.inf
        l[10] = math.nan
        t = torch.tensor([1, 2, 3, 0, 1, 0, 3, 4, 5, v - 1, 2, v], device="cuda")
        check(oz, l, t, 30)
        g = torch.Generator().manual_seed(7)
        dlp, dh, r = torch.randn(12, generator=g).cuda(), torch.randn(12, generator=g).cuda(), ref.rows(l)
        for a, b in ((dlp, None), (dlp, dh)):
            kw = dict(dentropy=b, entropy=None if b is None else r.entropy.float())
            got = oz.token_logprobs_backward(a, l, t, r.lse.float(), **kw)
            lin.assert_within(got, *ref.backward(l, t, a, b), f"dlogits {dt}")
            same = l.clone()
            oz.token_logprobs_backward(a, same, t, r.lse.float(), out=same, **kw)
            assert torch.equal(same.nan_to_num(7.0), got.nan_to_num(7.0))


def test_empty(oz):  # noqa: F811
    got = oz.token_logprobs(torch.empty(0, 9, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), top=3, entropy=True)
    assert got.lse.shape == got.logprobs.shape == got.entropy.shape == (0,) and got.top_tokens.shape == (0, 3)
    got = oz.token_logprobs(torch.empty(3, 0, device="cuda"), torch.tensor([-1, 0, 5], device="cuda"), entropy=True)
    assert (got.lse == -math.inf).all() and (got.entropy == 0).all() and got.logprobs[0] == 0 and torch.isnan(got.logprobs[1:]).all()


def test_nothing_beside_the_outputs_is_written(oz):  # noqa: F811
    for p, v in ((3, 13), (2, 9001), (1030, 777)):
        wide = torch.full((p + 2, v + 11), 7.0, device="cuda")
        out, l, t = wide[1:-1, 5:v + 5], normal(p, v, F32, 1), tokens_of(p, v, 2)
        got = oz.token_logprobs(l, t)
        d = torch.ones(p, device="cuda")
        want = oz.token_logprobs_backward(d, l, t, got.lse)
        oz.token_logprobs_backward(d, l, t, got.lse, out=out)
        assert torch.equal(out, want)
        out.fill_(7.0)
        assert (wide == 7).all()


def test_graph_and_streams(oz):  # noqa: F811
    l, t, d = normal(9, 50001, BF16, 1, 3.0), tokens_of(9, 50001, 1), torch.randn(9, device="cuda")

    def all_of(**kw):
        got = oz.token_logprobs(l, t, top=20, entropy=True, **kw)
        return (*got, oz.token_logprobs_backward(d, l, t, got.lse, dentropy=d, entropy=got.entropy, **kw))

    want = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = all_of(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of()
    for k in range(3):
        l.copy_(normal(9, 50001, BF16, 10 + k, 3.0))
        want = all_of()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_vocabulary_product_and_back(oz):  # noqa: F811
    """The norm, the vocabulary product, the log probabilities and all gradients, as a training step
    runs them, against autograd of the same step in 64 bits."""
    p, q, v = 150, 256, 5003
    x, r, w = normal(p, q, F16, 1), normal(p, q, F16, 2), (1 + 0.1 * normal(1, q, F16, 3)[0].float()).half()
    e, t = normal(v, q, F16, 4, 1 / 8), tokens_of(p, v, 5)
    dlp, dh = torch.randn(p, device="cuda") / p, 0.1 * torch.randn(p, device="cuda") / p
    y, h = oz.rms_norm(x, w, residual=r)
    logits = oz.linear(y, e)
    got = oz.token_logprobs(logits, t, entropy=True)
    scale = 1024.0  # the gradients, kept above f16's smallest
    d = oz.token_logprobs_backward(dlp * scale, logits, t, got.lse, dentropy=dh * scale, entropy=got.entropy)
    dy, de, _ = oz.linear_backward(d, y, e, needs=("x", "w"))
    dx, dw = oz.rms_norm_backward(dy, h, w)

    x64, w64, e64 = ((x.double() + r.double()).requires_grad_(), w.double().requires_grad_(), e.double().requires_grad_())
    y64 = x64 * (x64.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w64
    logp = torch.log_softmax(y64 @ e64.t(), 1)
    loss = (logp.gather(1, t.clamp(min=0)[:, None])[:, 0] * (t >= 0) * dlp.double()).sum() - (dh.double() * (logp.exp() * logp).sum(1)).sum()
    loss.backward()
    # four roundings to f16 lie between logits and dx (2^-11 each, relative in the norm); the logits, with magnitudes
    # up to 20, are themselves rounded to 2^-11 of that, which moves p by as much
    for a, b in ((dx, x64.grad), (dw, w64.grad), (de, e64.grad)):
        assert (a.double() / scale - b).norm() <= (4 + 20) * 2.0 ** -11 * b.norm()
