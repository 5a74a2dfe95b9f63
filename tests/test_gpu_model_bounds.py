"""The entry points of norm, adapters and log probabilities touch nothing beyond their arguments
(operands among NaN, outputs and the workspace among values that have to stay, the workspace full of
NaN at the start), leave operands and outputs of another stream's calls alone, can be captured on the
library's own buffer, and run together as a model's step has them."""
import pytest

from tests import adapters_reference as ad_ref
from tests import linear_plans as plans
from tests import linear_reference as lin
from tests import logprobs_reference as lp_ref
from tests import norm_reference as norm_ref
from tests.test_gpu_linear import BF16, F16, F32, normal, oz, torch, vector  # noqa: F401
from tests.test_gpu_linear_bounds import Place, Scratch, randn, stream

pytestmark = pytest.mark.gpu
TYPES = pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
NAN = float("nan")


def kind(oz, dtype):  # noqa: F811
    return {BF16: oz.OZ2_BF16, F16: oz.OZ2_F16, F32: oz.OZ2_F32}[dtype]


@pytest.mark.parametrize("p, q", [(1, 1), (3, 9), (5, 513), (600, 2047), (2, 8191), (520, 4100), (2, 32767)])
@TYPES
@pytest.mark.parametrize("pad", [0, 5])
def test_norm(oz, p, q, dtype, pad):  # noqa: F811
    k = kind(oz, dtype)
    x, r, w = Place(p, q, dtype, pad, NAN, randn(p, q, 1)), Place(p, q, dtype, pad, NAN, randn(p, q, 2)), Place(1, q, dtype, 0, NAN, randn(1, q, 3))
    h, y = Place(p, q, dtype, pad, 7.0), Place(p, q, dtype, pad, 7.0)
    assert oz.ozaki2_rms_norm(k, p, q, x.ptr, x.ld, r.ptr, r.ld, w.ptr, 1e-6, h.ptr, h.ld, y.ptr, y.ld, stream()) == oz.OZ2_OK
    want = norm_ref.hidden(x.view, r.view)
    assert torch.equal(h.view, want)
    lin.assert_within(y.view, *norm_ref.rms_norm(want, w.view[0], 1e-6), "y")
    levels, scale, h2 = Place(p, q, torch.int8, pad, -128), Place(1, p, F32, 0, 7.0), Place(p, q, dtype, pad, 7.0)
    assert oz.ozaki2_rms_norm_i8(k, p, q, x.ptr, x.ld, r.ptr, r.ld, w.ptr, 1e-6, h2.ptr, h2.ld, levels.ptr, levels.ld, scale.ptr, stream()) == oz.OZ2_OK
    assert torch.equal(h2.view, want) and (levels.view.abs().amax(1) == 127).all()
    dy, dh = Place(p, q, dtype, pad, NAN, randn(p, q, 4)), Place(p, q, dtype, pad, NAN, randn(p, q, 5))
    dx, dw, work = Place(p, q, dtype, pad, 7.0), Place(1, q, dtype, 0, 7.0), Scratch(oz.ozaki2_rms_norm_bwd_workspace_size(k, p, q))
    hin = Place(p, q, dtype, pad, NAN, want)
    rc = oz.ozaki2_rms_norm_bwd(k, p, q, dy.ptr, dy.ld, hin.ptr, hin.ld, w.ptr, 1e-6, dh.ptr, dh.ld, dx.ptr, dx.ld, dw.ptr, work.ptr, work.size, stream())
    assert rc == oz.OZ2_OK
    (wx, ww), (ex, ew) = norm_ref.backward(dy.view, hin.view, w.view[0], dh.view, 1e-6)
    lin.assert_within(dx.view, wx, ex, "dx")
    lin.assert_within(dw.view[0], ww, ew, "dw")
    for name, t in dict(x=x, r=r, w=w, h=h, y=y, levels=levels, scale=scale, h2=h2, dy=dy, dh=dh, hin=hin, dx=dx, dw=dw).items():
        t.check(name)
    work.check()


@pytest.mark.parametrize("sizes", [(1, 1, 1), (2, 17, 8), (16, 31, 17), (17, 65, 7), (65, 63, 129), (200, 77, 130)] + [s for s, _, _ in plans.FORWARD], ids=str)
@pytest.mark.parametrize("rank, count", [(8, 3), (13, 5), (80, 2)])
@pytest.mark.parametrize("pad", [0, 5])
def test_adapters(oz, sizes, rank, count, pad):  # noqa: F811
    (p, q, r), dtype = sizes, (BF16 if rank == 13 else F16)
    print("adapters", sizes, rank, pad, flush=True)
    x, w = Place(p, q, dtype, pad, NAN, randn(p, q, 1)), Place(r, q, dtype, pad, NAN, randn(r, q, 2, q ** -0.5))
    a, b = Place(count * rank, q, dtype, pad, NAN, randn(count * rank, q, 3, q ** -0.5)), Place(count * r, rank, dtype, pad, NAN, randn(count * r, rank, 4, rank ** -0.5))
    bias, res, y = Place(1, r, dtype, 0, NAN, randn(1, r, 5)), Place(p, r, dtype, pad, NAN, randn(p, r, 6)), Place(p, r, dtype, pad, 7.0)
    index = Place(1, p, torch.int32, 0, 0, (torch.arange(p, device="cuda") * 7 // 3 % (count + 2) - 1))
    scale = Place(1, count, F32, 0, NAN, torch.arange(1, count + 1, device="cuda")[None] / 2)
    aligned = 1 if pad == 0 and q % 8 == 0 else 0
    work = Scratch(oz.ozaki2_linear_adapters_workspace_size(kind(oz, dtype), p, q, r, count, rank, aligned))
    ad = oz.OZ2Adapters(count, rank, a.ptr, a.ld, rank * a.ld, b.ptr, b.ld, r * b.ld, index.ptr, scale.ptr)
    rc = oz.ozaki2_linear_adapters(kind(oz, dtype), p, q, r, x.ptr, x.ld, w.ptr, w.ld, bias.ptr, oz.OZ2_ACT_SILU, ad, res.ptr, res.ld,
                                   y.ptr, y.ld, work.ptr, work.size, stream())
    assert rc == oz.OZ2_OK
    want, bound = ad_ref.linear_adapters(x.view, w.view, a.view.unflatten(0, (count, rank)), b.view.unflatten(0, (count, r)),
                                         index.view[0], scale.view[0], bias.view[0], "silu", res.view)
    lin.assert_within(y.view, want, bound, "y")
    for name, t in dict(x=x, w=w, a=a, b=b, bias=bias, res=res, y=y, index=index, scale=scale).items():
        t.check(name)
    work.check()


@pytest.mark.parametrize("p, v", [(1, 1), (3, 13), (2, 4097), (9, 50003), (1030, 777)])
@TYPES
@pytest.mark.parametrize("pad", [0, 5])
def test_logprobs(oz, p, v, dtype, pad):  # noqa: F811
    k, top = kind(oz, dtype), min(v, 20)
    logits = Place(p, v, dtype, pad, NAN, randn(p, v, 1, 3.0))
    tokens = Place(1, p, torch.int64, 0, -9, torch.randint(0, v, (1, p), device="cuda"))
    lp, lse, h = (Place(1, p, F32, 0, 7.0) for _ in range(3))
    which, best = Place(p, top, torch.int64, 0, 7), Place(p, top, F32, 0, 7.0)
    which, best = (Place(1, p * top, t, 0, 7) for t in (torch.int64, F32))
    work = Scratch(oz.ozaki2_token_logprobs_workspace_size(p, v, top))
    rc = oz.ozaki2_token_logprobs(k, p, v, logits.ptr, logits.ld, tokens.ptr, top, lp.ptr, lse.ptr, h.ptr, which.ptr, best.ptr, work.ptr, work.size, stream())
    assert rc == oz.OZ2_OK
    r = lp_ref.rows(logits.view)
    lin.assert_within(lp.view[0], *lp_ref.given(r, tokens.view[0]), "logprob")
    assert torch.equal(which.view.view(p, top), lp_ref.largest(logits.view, top))
    dlp, dh, d = Place(1, p, F32, 0, NAN, randn(1, p, 2)), Place(1, p, F32, 0, NAN, randn(1, p, 3)), Place(p, v, dtype, pad, 7.0)
    rc = oz.ozaki2_token_logprobs_bwd(k, p, v, dlp.ptr, logits.ptr, logits.ld, tokens.ptr, lse.ptr, dh.ptr, h.ptr, d.ptr, d.ld, stream())
    assert rc == oz.OZ2_OK
    want, bound = lp_ref.backward(logits.view, tokens.view[0], dlp.view[0], dh.view[0])
    # (lse and the entropy are the forward call's own here, off by its error)
    more = (dlp.view[0].abs() + dh.view[0].abs() * (r.entropy + 30)).double()[:, None] * (r.d - r.logs[:, None]).exp() * (2 * r.err[:, None])
    more = more + dh.view[0].abs().double()[:, None] * (r.d - r.logs[:, None]).exp() * r.err_h[:, None]
    lin.assert_within(d.view, want, bound + more, "dlogits")
    for name, t in dict(logits=logits, tokens=tokens, lp=lp, lse=lse, h=h, which=which, best=best, dlp=dlp, dh=dh, d=d).items():
        t.check(name)
    work.check()


def calls(oz):  # noqa: F811
    """Operands by name, and a call on them, of each function."""
    torch.manual_seed(1)
    new = lambda *s: torch.randn(*s, device="cuda").half()  # noqa: E731
    index = lambda n, p: torch.randint(-1, n, (p,), device="cuda", dtype=torch.int32)  # noqa: E731
    tok = lambda v, p: torch.randint(0, v, (p,), device="cuda")  # noqa: E731
    return {
        "rms_norm": (lambda: dict(x=new(900, 700), weight=new(700), residual=new(900, 700)), oz.rms_norm),
        "rms_norm_i8": (lambda: dict(x=new(900, 700), weight=new(700), residual=new(900, 700)), oz.rms_norm_i8),
        "rms_norm_backward": (lambda: dict(dy=new(900, 700), h=new(900, 700), weight=new(700), dh=new(900, 700)), oz.rms_norm_backward),
        "linear_adapters": (lambda: dict(x=new(700, 512), w=new(600, 512), a=new(5, 16, 512), b=new(5, 600, 16), index=index(5, 700),
                                         scale=torch.ones(5, device="cuda"), bias=new(600), residual=new(700, 600)), oz.linear_adapters),
        "token_logprobs": (lambda: dict(logits=new(30, 40000), tokens=tok(40000, 30), top=5, entropy=True), oz.token_logprobs),
        "token_logprobs_backward": (lambda: dict(dlogprobs=torch.ones(30, device="cuda"), logits=new(30, 40000), tokens=tok(40000, 30),
                                                 lse=torch.full((30,), 11.0, device="cuda")), oz.token_logprobs_backward),
    }


@pytest.mark.parametrize("name", ["rms_norm", "rms_norm_i8", "rms_norm_backward", "linear_adapters", "token_logprobs", "token_logprobs_backward"])
def test_operands_dropped_after_a_call_on_a_stream(oz, name):  # noqa: F811
    make, call = calls(oz)[name]
    operands = make()
    flat = lambda t: t if isinstance(t, tuple) else (t,)  # noqa: E731
    want = [t.clone() for t in flat(call(**operands))]
    s, busy = torch.cuda.Stream(), torch.randn(8192, 8192, device="cuda")
    torch.mm(busy, busy)
    tensors = {k: t for k, t in operands.items() if torch.is_tensor(t)}
    places = {t.data_ptr() for t in tensors.values()}
    shapes = [(t.shape, t.dtype) for t in tensors.values()]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(8):
            torch.mm(busy, busy)
    got = call(**operands, stream=s)
    del operands, tensors
    assert not s.query(), "the stream is still busy before the call"
    others = [torch.full(shape, 77, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(2)]
    assert not places & {t.data_ptr() for t in others}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(flat(got), want))


def test_graph_on_the_librarys_buffer(oz):  # noqa: F811
    """Calls without a caller's scratch, captured on the library's buffer and replayed with larger eager
    calls, which take another, between the replays."""
    assert oz.ozaki2_release() == oz.OZ2_OK

    def step(p, q, dy, h, dx, dw, logits, lse, best, which, x, w, a, b, index, y):
        s = torch.cuda.current_stream().cuda_stream
        assert oz.ozaki2_rms_norm_bwd(oz.OZ2_F16, p, q, dy.data_ptr(), q, h.data_ptr(), q, None, 1e-6, None, q, dx.data_ptr(), q,
                                      dw.data_ptr(), None, 0, s) == oz.OZ2_OK
        v = logits.shape[1]
        assert oz.ozaki2_token_logprobs(oz.OZ2_F16, 3, v, logits.data_ptr(), v, None, 7, None, lse.data_ptr(), None, which.data_ptr(),
                                        best.data_ptr(), None, 0, s) == oz.OZ2_OK
        ad = oz.OZ2Adapters(4, 8, a.data_ptr(), q, 8 * q, b.data_ptr(), 8, 96 * 8, index.data_ptr(), None)
        assert oz.ozaki2_linear_adapters(oz.OZ2_F16, p, q, 96, x.data_ptr(), q, w.data_ptr(), q, None, 0, ad, None, 96, y.data_ptr(), 96,
                                         None, 0, s) == oz.OZ2_OK

    def operands(p, q, v, seed):
        new = lambda *s: normal(s[0], s[1], F16, seed + s[1])  # noqa: E731
        return [p, q, new(p, q), new(p, q) * 2, torch.empty(p, q, dtype=F16, device="cuda"), torch.empty(q, dtype=F16, device="cuda"),
                new(3, v), torch.empty(3, device="cuda"), torch.empty(3, 7, device="cuda"), torch.empty(3, 7, dtype=torch.int64, device="cuda"),
                new(p, q) * 0.5, new(96, q), new(32, q), new(4 * 96, 8), torch.arange(p, device="cuda", dtype=torch.int32) % 4,
                torch.empty(p, 96, dtype=F16, device="cuda")]

    small = operands(200, 512, 20000, 1)
    outs = (4, 5, 7, 8, 9, 15)
    step(*small)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*small)
    for k in range(3):
        large = operands(700 * (k + 1), 1024, 200000, 10 + k)
        step(*large)
        for i in (2, 3, 6, 10):
            small[i].copy_(normal(*small[i].shape, F16, 30 + k + i))
        step(*small)
        want = [small[i].clone() for i in outs]
        for i in outs:
            small[i].fill_(0)
        filled = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(small[i], w) for i, w in zip(outs, want)) and (filled == 0xFF).all()
    del graph
    assert oz.ozaki2_release() == oz.OZ2_OK


@pytest.mark.parametrize("p", [1, 6, 40])
def test_serving_step(oz, p):  # noqa: F811
    """Norm, int8 product, adapters, norm, vocabulary product and log probabilities as a serving
    step runs them, each stage against its 64-bit form on the stage's own operands."""
    q, r, v, n, k = 512, 1024, 4099, 6, 16
    stream_in, attn = normal(p, q, BF16, 1), normal(p, q, BF16, 2)
    g1, g2 = vector(q, BF16, 3), vector(q, BF16, 4)
    up, t_up = oz.quantize_rows(normal(r, q, F32, 5, q ** -0.5))
    down, a, b = normal(q, r, BF16, 6, r ** -0.5), normal(n * k, r, BF16, 7, r ** -0.5).view(n, k, r), normal(n * q, k, BF16, 8, 0.2).view(n, q, k)
    index, vocab = torch.arange(p, device="cuda", dtype=torch.int32) * 5 % (n + 1) - 1, normal(v, q, BF16, 9, q ** -0.5)
    levels, scale, h = oz.rms_norm_i8(attn, g1, residual=stream_in)
    assert torch.equal(h, norm_ref.hidden(attn, stream_in))
    up_out = oz.linear_i8(levels, up, t_up, activation="silu", x_scale=scale, dtype=BF16)
    z = (levels.double() @ up.double().t()) * scale.double()[:, None] * t_up.double()
    want = lin.activate(z, "silu")
    lin.assert_within(up_out, want, 2.0 ** -20 * (1 + z.abs()) * 2 + lin.rounding(want, BF16), "int8 product")
    out = oz.linear_adapters(up_out, down, a, b, index, residual=h)
    lin.assert_within(out, *ad_ref.linear_adapters(up_out, down, a, b, index, residual=h), "adapters")
    y = oz.rms_norm(out, g2)
    lin.assert_within(y, *norm_ref.rms_norm(out, g2, 1e-6), "norm")
    logits = oz.linear(y, vocab)
    got, rows = oz.token_logprobs(logits, top=20, entropy=True), lp_ref.rows(logits)
    which = lp_ref.largest(logits, 20)
    assert torch.equal(got.top_tokens, which)
    lin.assert_within(got.top_logprobs, *lp_ref.top_values(rows, which), "top_logprobs")
    again = oz.token_logprobs(logits, which[:, 0].contiguous())
    lin.assert_within(again.logprobs, *lp_ref.given(rows, which[:, 0]), "logprobs")
