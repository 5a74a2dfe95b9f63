"""The norm on the GPU against its 64-bit forms (tests/norm_reference.py, which derives the
bounds): lengths around every vector and thread-group edge, types, strides, in place, values at
the ends of the types' ranges, streams and graphs, and int8 rows into the int8 product."""
import pytest

from tests import linear_reference as lin
from tests import norm_reference as ref
from tests.test_gpu_linear import BF16, F16, F32, normal, oz, torch, vector  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = {"bf16": BF16, "f16": F16, "f32": F32}
SHAPES = [(1, 1), (3, 7), (2, 8), (5, 9), (1, 63), (700, 64), (513, 515), (4, 2047), (600, 2048), (1, 2048), (3, 2049), (520, 2056),
          (7, 8191), (1, 8192), (515, 8192), (2, 8193), (3, 32761), (1, 32768), (530, 12288)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("type", list(TYPES))
def test_norm(oz, shape, type):  # noqa: F811
    (p, q), dt = shape, TYPES[type]
    for k, (residual, weight, pad, shift) in enumerate([(True, True, 0, 0), (False, True, 3, 1), (True, False, 8, 0)]):
        print("norm", shape, type, residual, weight, pad, flush=True)
        x, r = normal(p, q, dt, k, pad=pad, shift=shift), normal(p, q, dt, 10 + k, 3.0, pad=pad) if residual else None
        w, eps = vector(q, dt, 20 + k) if weight else None, [1e-6, 1e-5, 0.5][k]
        h = ref.hidden(x, r)
        got = oz.rms_norm(x, w, residual=r, eps=eps)
        y, bound = ref.rms_norm(h, w, eps)
        if residual:
            assert torch.equal(got[1], h)
        lin.assert_within(got[0] if residual else got, y, bound, "y")
        got = oz.rms_norm_i8(x, w, residual=r, eps=eps)
        if residual:
            assert torch.equal(got[2], h)
        check_levels(got[0], got[1], *ref.norm(h, w, eps))


def check_levels(levels, scale, y, err):
    step = y.abs().amax(1) / 127
    lin.assert_within(scale, step, 50 * ref.U * step, "scale")
    assert (levels.abs().amax(1) == torch.where(step > 0, 127, 0)).all()
    # half a step, and what y is off by itself, scale and the product with its reciprocal
    assert ((levels.double() * scale.double()[:, None] - y).abs() <= 0.5 * step[:, None] + 2 * err + 60 * ref.U * y.abs()).all()


@pytest.mark.parametrize("shape", SHAPES + [(2100, 40), (1030, 2100)], ids=str)
@pytest.mark.parametrize("type", list(TYPES))
def test_backward(oz, shape, type):  # noqa: F811
    (p, q), dt = shape, TYPES[type]
    for k, (stream, weight, pad, shift) in enumerate([(True, True, 0, 0), (False, True, 3, 1), (True, False, 8, 0)]):
        print("backward", shape, type, stream, weight, pad, flush=True)
        h, dy = normal(p, q, dt, k, 2.0, pad=pad, shift=shift), normal(p, q, dt, 10 + k, pad=pad)
        dh = normal(p, q, dt, 20 + k, pad=pad, shift=shift) if stream else None
        w = vector(q, dt, 30 + k) if weight else None
        got = oz.rms_norm_backward(dy, h, w, dh=dh, eps=1e-5)
        (dx, dw), (ex, ew) = ref.backward(dy, h, w, dh, 1e-5)
        lin.assert_within(got[0], dx, ex, "dx")
        lin.assert_within(got[1], dw, ew, "dw")
        again = oz.rms_norm_backward(dy, h, w, dh=dh, eps=1e-5)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        one, none = oz.rms_norm_backward(dy, h, w, dh=dh, eps=1e-5, needs=("x",))
        assert none is None and torch.equal(one, got[0])
        none, one = oz.rms_norm_backward(dy, h, w, dh=dh, eps=1e-5, needs=("weight",))
        assert none is None and torch.equal(one, got[1])


def test_empty(oz):  # noqa: F811
    for p, q in ((0, 8), (3, 0), (0, 0)):
        x = torch.empty(p, q, dtype=BF16, device="cuda")
        y, h = oz.rms_norm(x, residual=x)
        assert y.shape == h.shape == (p, q)
        levels, scale = oz.rms_norm_i8(x)
        assert levels.shape == (p, q) and scale.shape == (p,) and (scale == 0).all()
        dx, dw = oz.rms_norm_backward(x, x)
        assert dx.shape == (p, q) and dw.shape == (q,) and (dw == 0).all()


@pytest.mark.parametrize("q", [64, 2500, 9000])
def test_ends_of_the_range(oz, q):  # noqa: F811
    """Rows of huge, tiny and zero values, and rows that hold infinities or NaN beside finite rows."""
    for dt in (BF16, F32):
        h = normal(8, q, dt, 1).clone()
        h[0] = 3e38 * torch.sign(h[0].float())
        h[1] *= 1e25
        h[2] *= 1e-30
        h[3] = 0
        h[4, q // 2] = float("inf")
        h[5, q - 1] = float("nan")
        w = vector(q, dt, 2)
        y, bound = ref.rms_norm(h, w, 1e-6)
        lin.assert_within(oz.rms_norm(h, w), y, bound, f"y {dt}")
        levels, scale = oz.rms_norm_i8(h, w)
        finite = torch.tensor([0, 1, 6, 7], device="cuda")
        check_levels(levels[finite], scale[finite], *(t[finite] for t in ref.norm(h, w, 1e-6)))
        assert scale[3] == 0 and (levels[3:6] == 0).all() and torch.isnan(scale[4:6]).all()
        dy, finite = normal(8, q, dt, 3), torch.tensor([0, 1, 2, 3, 6, 7], device="cuda")
        got = oz.rms_norm_backward(dy, h, w, needs=("x",))[0]
        (dx, _), (ex, _) = ref.backward(dy, h, w, None, 1e-6)
        lin.assert_within(got[finite], dx[finite], ex[finite] + 2.0 ** -126, f"dx {dt}")
        # gradients times values past f32's range, neither of them near it
        big = (dy.float() * 1e22).to(dt)
        h2 = (normal(8, q, dt, 4).float() * 1e18).to(dt)
        got = oz.rms_norm_backward(big, h2, w)
        (dx, dw), (ex, ew) = ref.backward(big, h2, w, None, 1e-6)
        lin.assert_within(got[0], dx, ex, f"dx of large gradients {dt}")
        lin.assert_within(got[1], dw, ew, f"dw of large gradients {dt}")


def test_in_place(oz):  # noqa: F811
    x, r, w = normal(300, 1000, F16, 1, pad=4), normal(300, 1000, F16, 2), vector(1000, F16, 3)
    y, h = oz.rms_norm(x, w, residual=r)
    for out, hidden in (("x", "r"), ("r", "x"), (None, "r"), ("x", None)):
        t = {"x": x.clone(), "r": r.clone(), None: None}
        got = oz.rms_norm(t["x"], w, residual=t["r"], out=t[out], hidden=t[hidden])
        assert torch.equal(got[0], y) and torch.equal(got[1], h)
        assert out is None or got[0] is t[out]
        assert hidden is None or got[1] is t[hidden]
    with pytest.raises(oz.Oz2Error):
        oz.rms_norm(x, w, residual=r, out=r, hidden=r)
    before = r._version
    oz.rms_norm_i8(x, w, residual=r, hidden=r)
    assert torch.equal(r, h) and r._version > before


def test_nothing_beside_the_outputs_is_written(oz):  # noqa: F811
    for dt in (BF16, F32):
        for p, q in ((3, 13), (600, 2047), (2, 8195)):
            wide = torch.full((p + 2, q + 11), 7.0, dtype=dt, device="cuda")
            out = wide[1:-1, 5:q + 5]
            x, r = normal(p, q, dt, 1), normal(p, q, dt, 2)
            y, h = oz.rms_norm(x, residual=r)
            oz.rms_norm(x, residual=r, out=out)
            assert torch.equal(out, y)
            out.fill_(7.0)
            assert (wide == 7).all()
            oz.rms_norm(x, residual=r, hidden=out)
            assert torch.equal(out, h)
            out.fill_(7.0)
            assert (wide == 7).all()


def test_graph_and_streams(oz):  # noqa: F811
    """Captured calls replayed on new inputs, eager ones between the replays; a call on a stream."""
    x, r, w, dy = normal(700, 1000, BF16, 1), normal(700, 1000, BF16, 2), vector(1000, BF16, 3), normal(700, 1000, BF16, 4)

    def all_of(**kw):
        y, h = oz.rms_norm(x, w, residual=r, **kw)
        return (y, h, *oz.rms_norm_i8(x, w, residual=r, **kw), *oz.rms_norm_backward(dy, h, w, dh=r, **kw))

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
        x.copy_(normal(700, 1000, BF16, 10 + k))
        dy.copy_(normal(700, 1000, BF16, 20 + k))
        want = all_of()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def product_of_levels(levels, s, v, t, bias, residual):
    """(y, bound) of residual + gelu(s t (levels v^T) + bias): the integer sums are exact, the two
    scalings, their conversion and the bias round four times, gelu's slope is at most 1.13."""
    a = (levels.double() @ v.double().t()) * s.double()[:, None] * t.double()
    err = 4 * ref.U * a.abs()
    a = a + bias.double()
    err = err + 2 * ref.U * a.abs()
    y = lin.activate(a, "gelu") + residual.double()
    return y, (1.2 * err + 2.0 ** -20 * (1 + a.abs()) + 2 * ref.U * y.abs()) * 1.01 + lin.rounding(y, bias.dtype)


@pytest.mark.parametrize("p, q, r", [(1, 200, 72), (2, 4096, 500), (7, 1001, 64), (16, 300, 33), (40, 515, 130), (300, 2048, 513)])
def test_levels_into_the_product(oz, p, q, r):  # noqa: F811
    """int8 rows of the norm through the int8 product: the same bits as a product that quantises the
    same rows itself, and within the bound of the norm's values."""
    for dt in (BF16, F16):
        x, g = normal(p, q, dt, 1), vector(q, dt, 2)
        v, t = oz.quantize_rows(normal(r, q, F32, 3, q ** -0.5))
        b, res = vector(r, dt, 4), normal(p, r, dt, 5)
        levels, s = oz.quantize_rows(x)
        kw = dict(bias=b, activation="gelu", residual=res)
        want = oz.linear_i8(x, v, t, **kw)
        assert torch.equal(oz.linear_i8(levels, v, t, x_scale=s, dtype=dt, **kw), want)
        wide = torch.zeros(p, q + 3, dtype=torch.int8, device="cuda")
        wide[:, :q] = levels
        assert torch.equal(oz.linear_i8(wide[:, :q], v, t, x_scale=s, dtype=dt, **kw), want)
        levels, s = oz.rms_norm_i8(x, g)
        y, bound = product_of_levels(levels, s, v, t, b, res)
        lin.assert_within(oz.linear_i8(levels, v, t, x_scale=s, dtype=dt, **kw), y, bound, "norm into the product")
