"""The product with adapters on the GPU against its 64-bit form (tests/adapters_reference.py, which
derives the bounds): every kernel the plan chooses from, ranks around every block edge, rows without
an adapter, requests in and out of order, strides, infinities in one request's adapter, streams
and graphs."""
import pytest

from tests import adapters_reference as ref
from tests import linear_plans as plans
from tests import linear_reference as lin
from tests.test_gpu_linear import BF16, F16, normal, oz, torch, vector  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = {"bf16": BF16, "f16": F16}


def indices(p, n, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "mixed":       # every row its own, some without (-1, n and beyond)
        return torch.randint(-1, n + 1, (p,), generator=g).to(torch.int32).cuda()
    if kind == "requests":    # a few long requests
        cuts = torch.randint(0, p + 1, (3,), generator=g).sort().values
        return torch.randint(-1, n, (4,), generator=g)[torch.searchsorted(cuts, torch.arange(p), right=True)].to(torch.int32).cuda()
    return torch.full((p,), n - 1 if kind == "one" else -1, dtype=torch.int32).cuda()


def operands(p, q, r, n, k, dt, seed, pad=0, shift=0):
    x, w = normal(p, q, dt, seed, pad=pad, shift=shift), normal(r, q, dt, seed + 1, max(q, 1) ** -0.5, pad=pad, shift=shift)
    a = normal(n * k, q, dt, seed + 2, max(q, 1) ** -0.5, pad=pad).unflatten(0, (n, k))
    b = normal(n * r, k, dt, seed + 3, max(k, 1) ** -0.5, pad=pad, shift=shift).unflatten(0, (n, r))
    return x, w, a, b


SHAPES = [  # p, q, r, n, k
    (1, 64, 8, 1, 1), (1, 2048, 515, 5, 16), (2, 300, 100, 3, 8), (3, 7, 5, 2, 3), (8, 4096, 200, 20, 33), (9, 1000, 72, 4, 64),
    (16, 512, 4096, 9, 65), (16, 8192, 64, 16, 16), (17, 33, 65, 2, 12), (37, 2048, 256, 40, 32), (64, 64, 64, 64, 8), (65, 127, 129, 7, 24),
    (100, 1024, 250, 5, 100), (130, 256, 257, 3, 17), (300, 1000, 77, 11, 5), (513, 72, 511, 6, 128), (700, 1344, 1100, 4, 256),
    (2049, 512, 2100, 3, 64),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("type", list(TYPES))
def test_adapters(oz, shape, type):  # noqa: F811
    (p, q, r, n, k), dt = shape, TYPES[type]
    options = [("mixed", "none", False, False, False, 0, 0), ("requests", "gelu", True, True, True, 8, 8),
               ("one", "silu", True, False, True, 3, 1), ("none", "relu", False, True, False, 0, 0)]
    for i, (kind, act, bias, residual, scaled, pad, shift) in enumerate(options):
        print("adapters", shape, type, kind, pad, shift, flush=True)
        x, w, a, b = operands(p, q, r, n, k, dt, 10 * i, pad, shift)
        index = indices(p, n, kind, i)
        scale = torch.rand(n, device="cuda") * 2 if scaled else None
        bias = vector(r, dt, 70) if bias else None
        res = normal(p, r, dt, 80, pad=pad) if residual else None
        got = oz.linear_adapters(x, w, a, b, index, scale=scale, bias=bias, activation=act, residual=res)
        y, bound = ref.linear_adapters(x, w, a, b, index, scale, bias, act, res)
        lin.assert_within(got, y, bound, f"y {kind}")
        if kind == "none":
            assert torch.equal(got, oz.linear(x, w, bias=bias, activation=act, residual=res))
        assert torch.equal(oz.linear_adapters(x, w, a, b, index, scale=scale, bias=bias, activation=act, residual=res), got)


@pytest.mark.parametrize("sizes, tile, split", plans.FORWARD, ids=str)
def test_every_kernel(oz, sizes, tile, split):  # noqa: F811
    """Every kernel that the plan chooses from, and infinities in one adapter, which stay in its own
    rows."""
    p, q, r = sizes
    assert plans.kernel(plans.forward(p, q, r)) == (tile, split)
    rows = f"{tile} {sizes}"
    for dt in TYPES.values():
        print("kernel", rows, dt, flush=True)
        x, w, a, b = operands(p, q, r, 6, 40, dt, 5)
        index = indices(p, 6, "mixed", 3)
        y, bound = ref.linear_adapters(x, w, a, b, index)
        want = oz.linear_adapters(x, w, a, b, index)
        lin.assert_within(want, y, bound, rows)
        b[2, 5:9, 3] = float("inf")
        a[4, 1, 7] = float("nan")
        b[5] = float("-inf")
        got = oz.linear_adapters(x, w, a, b, index)
        clean = (index != 2) & (index != 4) & (index != 5)
        assert torch.equal(got[clean], want[clean])
        if bool((index == 4).any()):
            assert torch.isnan(got[index == 4]).all()
        two = index == 2
        if bool(two.any()):
            assert torch.equal(got[two][:, :5], want[two][:, :5]) and torch.equal(got[two][:, 9:], want[two][:, 9:])
            assert not torch.isfinite(got[two][:, 5:min(9, r)]).any()


@pytest.mark.parametrize("p", [1, 5, 16, 40, 300])
def test_strides(oz, p):  # noqa: F811
    """Adapters inside larger buffers, one matrix shared by all, and without any."""
    q, r, n, k = 200, 136, 4, 8
    x, w, _, _ = operands(p, q, r, 1, 1, BF16, 1)
    a, b = normal(n * 12, q + 24, BF16, 2).view(n, 12, q + 24)[:, 2:10, 8:208], normal(n * r, 64, BF16, 3).view(n, r, 64)[:, :, 16:24]
    index = indices(p, n, "mixed", p)
    for aa, bb in ((a, b), (a[:1].expand(n, k, q), b), (a, b[:1].expand(n, r, k)), (a.clone()[1:2], b[1:2])):
        y, bound = ref.linear_adapters(x, w, aa, bb, index)
        lin.assert_within(oz.linear_adapters(x, w, aa, bb, index), y, bound, "strided")
    plain = oz.linear(x, w)
    for n, k in ((0, 8), (4, 0)):
        none = torch.empty(n, k, q, dtype=BF16, device="cuda"), torch.empty(n, r, k, dtype=BF16, device="cuda")
        assert torch.equal(oz.linear_adapters(x, w, *none, index), plain)


def test_empty(oz):  # noqa: F811
    for p, q, r in ((0, 16, 8), (3, 16, 0), (3, 0, 8), (40, 0, 70)):
        x, w, a, b = operands(p, q, r, 2, 4, F16, 1)
        got = oz.linear_adapters(x, w, a, b, torch.zeros(p, dtype=torch.int32, device="cuda"))
        assert got.shape == (p, r) and (got == 0).all()
    with pytest.raises(oz.Oz2Error):
        x, w, a, b = operands(3, 16, 8, 2, 257, F16, 1)
        oz.linear_adapters(x, w, a, b, torch.zeros(3, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("p, q, r", [(2, 200, 72), (40, 515, 130), (600, 512, 515)])
def test_graph_streams_and_in_place(oz, p, q, r):  # noqa: F811
    x, w, a, b = operands(p, q, r, 5, 16, F16, 1)
    index, res = indices(p, 5, "mixed", 1), normal(p, r, F16, 9)
    call = lambda **kw: oz.linear_adapters(x, w, a, b, index, activation="gelu", residual=res, **kw)  # noqa: E731
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    wide = torch.full((p + 2, r + 9), 7.0, dtype=F16, device="cuda")
    out = wide[1:-1, 3:r + 3]
    assert call(out=out) is out and torch.equal(out, want)
    out.fill_(7.0)
    assert (wide == 7).all()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for k in range(3):
        x.copy_(normal(p, q, F16, 20 + k))
        index.copy_(indices(p, 5, "mixed", 30 + k))
        want = call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    keep = res.clone()
    got = oz.linear_adapters(x, w, a, b, index, activation="gelu", residual=keep, out=keep)
    assert got is keep and torch.equal(keep, want)
