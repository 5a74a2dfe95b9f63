"""The linear-layer entry points touch nothing beyond their arguments: every operand lies among NaN
(int8: -128), every output and the workspace, of exactly the size asked for, among values that have
to stay, and the workspace starts full of NaN."""
import pytest

from tests import linear_plans as plans
from tests import linear_reference as ref
from tests.test_gpu_linear import BF16, F16, oz, torch  # noqa: F401

pytestmark = pytest.mark.gpu
TYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
ODD = [(1, 1, 1), (1, 7, 9), (2, 17, 8), (5, 64, 33), (16, 31, 17), (17, 65, 7), (64, 129, 127), (65, 63, 129), (200, 77, 130)]
MARGIN = 4096  # elements on either side


class Place:
    """A matrix (rows of cols, ld apart) or vector inside a buffer full of `fill`."""

    def __init__(self, rows, cols, dtype, pad, fill, values=None):
        self.ld, shift = cols + pad, MARGIN + (3 if pad % 8 else 0)
        if pad % 8 == 0:
            self.ld += -self.ld % 16      # rows on 16-byte boundaries in every type
        self.flat = torch.full((shift + rows * self.ld + MARGIN,), fill, dtype=dtype, device="cuda")
        self.view = self.flat[shift:shift + rows * self.ld].view(rows, self.ld)[:, :cols]
        if values is not None:
            self.view.copy_(values)
        self.before = self.flat.clone()

    @property
    def ptr(self):
        return self.view.data_ptr()

    def check(self, what):
        """Nothing but the matrix itself has changed."""
        shift = self.view.storage_offset()
        now, was = self.flat.clone(), self.before
        rows, cols = self.view.shape
        for t in (now, was):
            t[shift:shift + rows * self.ld].view(rows, self.ld)[:, :cols] = 0
        assert torch.equal(now.view(torch.uint8), was.view(torch.uint8)), f"written beside {what}"


class Scratch:
    def __init__(self, size):
        self.size = size
        self.flat = torch.full((size + 2 * MARGIN,), 0xFF, dtype=torch.uint8, device="cuda")
        self.start = -self.flat.data_ptr() % 256 + 1024
        self.flat[:self.start] = 0xA5
        self.flat[self.start + size:] = 0xA5

    @property
    def ptr(self):
        return self.flat.data_ptr() + self.start

    def check(self):
        assert (self.flat[:self.start] == 0xA5).all() and (self.flat[self.start + self.size:] == 0xA5).all(), "beside the workspace"


def randn(rows, cols, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, cols, generator=g, device="cuda") * scale


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("shape", ODD + [s for s, _, _ in plans.FORWARD], ids=str)
@TYPES
@pytest.mark.parametrize("pad", [0, 5])
def test_linear(oz, shape, dtype, pad):  # noqa: F811
    p, q, r = shape
    print("linear", shape, dtype, pad, flush=True)
    nan = float("nan")
    x, w = Place(p, q, dtype, pad, nan, randn(p, q, 1)), Place(r, q, dtype, pad, nan, randn(r, q, 2, q ** -0.5))
    b, res = Place(1, r, dtype, pad, nan, randn(1, r, 3)), Place(p, r, dtype, pad, nan, randn(p, r, 4))
    y, z = Place(p, r, dtype, pad, 7.0), Place(p, r, dtype, pad, 7.0)
    kind = oz.OZ2_BF16 if dtype is BF16 else oz.OZ2_F16
    aligned = oz.OZ2_LINEAR_ALIGNED if pad == 0 and q % 8 == 0 else 0
    work = Scratch(oz.ozaki2_linear_workspace_size(oz.OZ2_LINEAR_FWD | aligned, kind, p, q, r))
    rc = oz.ozaki2_linear(kind, p, q, r, x.ptr, x.ld, w.ptr, w.ld, b.ptr, oz.OZ2_ACT_SILU, oz.OZ2Dropout(0.1, 3, 4), res.ptr,
                          res.ld, z.ptr, z.ld, y.ptr, y.ld, work.ptr, work.size, stream())
    assert rc == oz.OZ2_OK
    wy, wz, ey, ez = ref.linear(x.view, w.view, b.view[0], "silu", res.view, (0.1, 3, 4))
    ref.assert_within(y.view, wy, ey, "y")
    ref.assert_within(z.view, wz, ez, "z")
    for name, t in dict(x=x, w=w, b=b, res=res, y=y, z=z).items():
        t.check(name)
    work.check()


@pytest.mark.parametrize("shape", ODD + [s for s, *_ in plans.BACKWARD], ids=str)
@TYPES
@pytest.mark.parametrize("pad", [0, 5])
def test_linear_backward(oz, shape, dtype, pad):  # noqa: F811
    p, q, r = shape
    nan = float("nan")
    kind = oz.OZ2_BF16 if dtype is BF16 else oz.OZ2_F16
    dy, x, w = (Place(*s, dtype, pad, nan, randn(*s, k)) for k, s in enumerate(((p, r), (p, q), (r, q))))
    z = Place(p, r, dtype, pad, nan, randn(p, r, 9))
    aligned = oz.OZ2_LINEAR_ALIGNED if pad == 0 and q % 8 == 0 else 0
    for act, drop in (("none", None), ("gelu", (0.1, 3, 4))):
        print("linear_bwd", shape, dtype, pad, act, flush=True)
        dx, dw, db = Place(p, q, dtype, pad, 7.0), Place(r, q, dtype, pad, 7.0), Place(1, r, dtype, pad, 7.0)
        work = Scratch(oz.ozaki2_linear_workspace_size(oz.OZ2_LINEAR_BWD | aligned, kind, p, q, r))
        rc = oz.ozaki2_linear_bwd(kind, p, q, r, dy.ptr, dy.ld, x.ptr, x.ld, w.ptr, w.ld, z.ptr if act != "none" else None, z.ld,
                                  oz.ACTIVATIONS[act], oz.OZ2Dropout(*drop) if drop else None, dx.ptr, dx.ld, dw.ptr, dw.ld,
                                  db.ptr, work.ptr, work.size, stream())
        assert rc == oz.OZ2_OK
        want, bound = ref.linear_backward(dy.view, x.view, w.view, z.view if act != "none" else None, act, drop)
        for name, g, v, e in zip(("dx", "dw", "db"), (dx.view, dw.view, db.view[0]), want, bound):
            ref.assert_within(g, v, e, name)
        for name, t in dict(dy=dy, x=x, w=w, z=z, dx=dx, dw=dw, db=db).items():
            t.check(name)
        work.check()


@pytest.mark.parametrize("shape", ODD + [s for s, _, _ in plans.INT8], ids=str)
@TYPES
@pytest.mark.parametrize("pad", [0, 5])
def test_linear_i8(oz, shape, dtype, pad):  # noqa: F811
    p, q, r = shape
    print("linear_i8", shape, dtype, pad, flush=True)
    nan = float("nan")
    levels, scales = ref.quantize(randn(r, q, 2, q ** -0.5))
    x, v = Place(p, q, dtype, pad, nan, randn(p, q, 1)), Place(r, q, torch.int8, pad, -128, levels)
    t, b = Place(1, r, torch.float32, pad, nan, scales[None]), Place(1, r, dtype, pad, nan, randn(1, r, 3))
    res, y = Place(p, r, dtype, pad, nan, randn(p, r, 4)), Place(p, r, dtype, pad, 7.0)
    kind = oz.OZ2_BF16 if dtype is BF16 else oz.OZ2_F16
    aligned = oz.OZ2_LINEAR_ALIGNED if pad == 0 and q % 16 == 0 else 0
    work = Scratch(oz.ozaki2_linear_workspace_size(oz.OZ2_LINEAR_I8 | aligned, kind, p, q, r))
    rc = oz.ozaki2_linear_i8(kind, p, q, r, x.ptr, x.ld, v.ptr, v.ld, t.ptr, b.ptr, oz.OZ2_ACT_GELU, res.ptr, res.ld, y.ptr, y.ld,
                             work.ptr, work.size, stream())
    assert rc == oz.OZ2_OK
    want, bound = ref.linear_i8(x.view, v.view, t.view[0], b.view[0], "gelu", res.view)
    ref.assert_within(y.view, want, bound, "y")
    for name, m in dict(x=x, v=v, t=t, b=b, res=res, y=y).items():
        m.check(name)
    work.check()


@pytest.mark.parametrize("shape", [(1, 1), (3, 9), (16, 2048), (33, 2047), (900, 515)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, F16, torch.float32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 5])
def test_rows(oz, shape, dtype, pad):  # noqa: F811
    p, r = shape
    nan = float("nan")
    kind = {BF16: oz.OZ2_BF16, F16: oz.OZ2_F16, torch.float32: oz.OZ2_F32}[dtype]
    x, res, y = Place(p, r, dtype, pad, nan, randn(p, r, 1)), Place(p, r, dtype, pad, nan, randn(p, r, 2)), Place(p, r, dtype, pad, 7.0)
    assert oz.ozaki2_dropout_add(kind, p, r, x.ptr, x.ld, res.ptr, res.ld, oz.OZ2Dropout(0.3, 5, 6), y.ptr, y.ld, stream()) == oz.OZ2_OK
    want = ref.dropped(x.view.double(), (0.3, 5, 6))[0] + res.view.double()
    ref.assert_within(y.view, want, ref.rounding(want, dtype) + 2.0 ** -22 * (want.abs() + res.view.double().abs()), "y")
    q, s = Place(p, r, torch.int8, pad, 55), Place(1, p, torch.float32, pad, 7.0)
    assert oz.ozaki2_quantize_rows(kind, p, r, x.ptr, x.ld, q.ptr, q.ld, s.ptr, stream()) == oz.OZ2_OK
    levels, scales = ref.quantize(x.view)
    assert torch.equal(q.view, levels) and torch.equal(s.view[0], scales)
    for name, m in dict(x=x, res=res, y=y, q=q, s=s).items():
        m.check(name)
