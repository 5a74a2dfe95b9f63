"""How the product with adapters holds S = scale X A^T between its two products: over the whole range
of f32 whatever the operands' type, with more bits than the operands have, and alike on every
kernel, so that a token's result does not depend on how many tokens are beside it.

Bounds.  S is summed and scaled in f32: off by at most (q + 34) 2^-23 of the magnitudes it is summed
from.  The tile kernels hold it as two terms of the operands' type.  With 2^e the power of two at or below
|S|: bf16's first term is S cut to 8 significant bits or one unit below, so the rest is at most 2^(e-7), and
rounding it to 8 bits moves it by at most 2^(e-16).  f16 likewise: a rest of at most 2^(e-10), moved by 2^(e-22), or,
where the rest is subnormal, by up to one of its steps of 2^-24, beside a largest magnitude of 2^13 at least
in each 64 elements of a row: 2^-22 of S and 2^-37 of that largest one.  The product with B adds at most two
times the rank and 64 terms, each in f32.
"""
import pytest

from tests import linear_plans as plans
from tests import linear_reference as lin
from tests.test_gpu_adapters import TYPES, indices
from tests.test_gpu_linear import BF16, F16, normal, oz, torch  # noqa: F401

pytestmark = pytest.mark.gpu

# p, q, r: one row and few, tiles of every size, the depth of S in parts and in one, cut rows and columns
SIZES = [(1, 512, 200), (5, 2048, 96), (16, 600, 130), (17, 512, 200), (40, 600, 130), (37, 4096, 264), (64, 96, 65), (300, 512, 200),
         (257, 2056, 33), (520, 640, 1032), (2049, 264, 2056)]


def reference(x, w, a, b, index, scale, residual=None):
    """(y, bound) in 64 bits."""
    dt, (q, k) = x.dtype, (x.shape[1], a.shape[1])
    y = x.double() @ w.double().t()
    err = (q + 16) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().t())
    for j in range(a.shape[0]):
        at = (index == j).nonzero()[:, 0]
        if len(at) == 0:
            continue
        xj, aj, bj, c = x[at].double(), a[j].double(), b[j].double(), scale[j].double()
        s = c * (xj @ aj.t())
        most = torch.cat([t.abs().amax(1, keepdim=True).expand_as(t) for t in s.split(64, 1)], 1)
        held = 2.0 ** -16 * s.abs() if dt == BF16 else 2.0 ** -22 * s.abs() + 2.0 ** -37 * most
        serr = c.abs() * (q + 34) * 2.0 ** -23 * (xj.abs() @ aj.abs().t()) + held
        y[at] += s @ bj.t()
        err[at] += 1.01 * (serr @ bj.abs().t()) + (2 * k + 64) * 2.0 ** -23 * (s.abs() @ bj.abs().t())
    err = err + 2.0 ** -23 * y.abs()
    if residual is not None:
        y = y + residual.double()
        err = err + 2.0 ** -23 * y.abs()
    return y, err * 1.01 + lin.rounding(y, dt)


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("k", [8, 40, 100])
@pytest.mark.parametrize("type", list(TYPES))
def test_range(oz, sizes, k, type):  # noqa: F811
    """Adapters whose S is far below and far above f16's range in one batch, by their scale and by
    their elements; B undoes it, and holds zeros, as a fresh adapter's does throughout."""
    (p, q, r), dt, n = sizes, TYPES[type], 7
    x, w = normal(p, q, dt, 1), normal(r, q, dt, 2, q ** -0.5)
    a, b = normal(n * k, q, dt, 3, q ** -0.5).view(n, k, q), normal(n * r, k, torch.float32, 4, k ** -0.5).view(n, r, k)
    scale = torch.tensor([1e6, 1e-6, 1.0, 3e7, 1e6, 2e-8, 0.0], device="cuda")
    a[3] *= 30
    b *= torch.tensor([1e-6, 2e4, 1.0, 1e-7, 0.0, 4e4, 1.0], device="cuda")[:, None, None]
    b[:, ::3, 1::2] = 0
    # S's elements of one row apart by 2^20 and more
    a[2, ::2] *= 512
    a[2, 1::2] /= 2048
    b = b.to(dt)
    index = indices(p, n, "mixed", p)
    if p < 8:
        for j in range(n):
            check(oz, x, w, a, b, torch.full_like(index, j), scale, j)
    check(oz, x, w, a, b, index, scale, "mixed")
    check(oz, x, w, a, b, indices(p, n, "requests", p + 1), scale, "requests")


def check(oz, x, w, a, b, index, scale, what):  # noqa: F811
    print("adapters' range", tuple(x.shape), tuple(b.shape), what, flush=True)
    got = oz.linear_adapters(x, w, a, b, index, scale=scale)
    y, bound = reference(x, w, a, b, index, scale)
    lin.assert_within(got, y, bound, f"y {what}")


@pytest.mark.parametrize("sizes", SIZES + [s for s, _, _ in plans.FORWARD], ids=str)
@pytest.mark.parametrize("type", list(TYPES))
def test_bits(oz, sizes, type):  # noqa: F811
    """The adapters' term alone, with a residual that takes all but its last bits away: what is left shows how
    many S was held in."""
    (p, q, r), dt, n = sizes, TYPES[type], 5
    for k in (16, 72):
        x, w = normal(p, q, dt, 1), torch.zeros(r, q, dtype=dt, device="cuda")
        a, b = normal(n * k, q, dt, 3, q ** -0.5).view(n, k, q), normal(n * r, k, dt, 4, k ** -0.5).view(n, r, k)
        index, scale = indices(p, n, "mixed", p), torch.rand(n, device="cuda") + 0.5
        y, _ = reference(x, w, a, b, index, scale)
        residual = -y.to(dt)
        print("adapters' bits", sizes, k, flush=True)
        got = oz.linear_adapters(x, w, a, b, index, scale=scale, residual=residual)
        y, bound = reference(x, w, a, b, index, scale, residual)
        lin.assert_within(got, y, bound, "y")


@pytest.mark.parametrize("p", [1, 16, 17, 64, 300, 2049])
@pytest.mark.parametrize("type", list(TYPES))
def test_infinities_keep_their_sign(oz, p, type):  # noqa: F811
    """An infinite element of A or B gives infinities of the term's sign, on few rows and on many."""
    dt, q, r, k = TYPES[type], 256, 520 if p < 2000 else 2056, 24
    x, w = normal(p, q, dt, 1), normal(r, q, dt, 2, q ** -0.5)
    a, b = normal(3 * k, q, dt, 3, q ** -0.5).view(3, k, q), normal(3 * r, k, dt, 4, k ** -0.5).view(3, r, k)
    b[b == 0] = 1
    b[0, 5, 3] = float("inf")
    b[0, r - 1, k - 1] = -float("inf")
    a[1, 7, 9] = float("inf")
    index = torch.arange(p, device="cuda", dtype=torch.int32) % 3
    for j in range(3 if p < 3 else 1):
        at = (index + j) % 3
        got = oz.linear_adapters(x, w, a, b, at).double()
        want = x.double() @ w.double().t()
        for i in range(3):
            rows = (at == i).nonzero()[:, 0]
            if len(rows):
                want[rows] += (x[rows].double() @ a[i].double().t()) @ b[i].double().t()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.isinf(got), torch.isinf(want)) and bool((got.sign() == want.sign())[torch.isinf(want)].all())


def test_a_token_alone_and_among_others(oz):  # noqa: F811
    """An f16 adapter past f16's range between the products: finite for one token, and as finite among many."""
    q, r, k = 256, 136, 16
    x = normal(40, q, F16, 1)
    w, a, b = normal(r, q, F16, 2, q ** -0.5), normal(k, q, F16, 3, q ** -0.5)[None], torch.zeros(1, r, k, dtype=F16, device="cuda")
    index, scale = torch.zeros(40, dtype=torch.int32, device="cuda"), torch.tensor([1e6], device="cuda")
    for p in (1, 8, 16, 17, 40):
        got = oz.linear_adapters(x[:p], w, a, b, index[:p], scale=scale)
        assert torch.equal(got, oz.linear(x[:p], w)), p  # B is all zeros: the product alone
