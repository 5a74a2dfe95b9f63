"""The linear-layer operators on the GPU against their 64-bit forms (tests/linear_reference.py,
which derives the bounds): sizes around every tile and vector edge, types, epilogues, row
strides and alignments, empty sizes, non-finite values, streams and graphs."""
import pytest

from tests import linear_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def oz():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    from fp64_gemm_emulation_amd import binding
    return binding


def normal(rows, cols, dtype, seed, scale=1.0, pad=0, shift=0):
    """rows x cols values, rows `pad` elements apart and the first `shift` elements into a buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.empty(shift + rows * (cols + pad), dtype=dtype, device="cuda")
    view = flat[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(torch.randn(rows, cols, generator=g, device="cuda") * scale)
    return view


def vector(n, dtype, seed):
    return normal(1, n, dtype, seed)[0]


# sizes around the edges of vectors (8), fragments (16, 32), tiles (64 to 256) and depth blocks
SHAPES = [(1, 1, 1), (1, 64, 8), (2, 8, 300), (3, 7, 5), (1, 2048, 515), (15, 96, 33), (16, 4096, 64), (17, 33, 65),
          (31, 640, 128), (33, 200, 1030), (64, 64, 64), (65, 127, 129), (100, 1024, 250), (128, 520, 128),
          (130, 256, 257), (257, 512, 640), (300, 1000, 77), (513, 72, 511), (700, 1344, 1100), (1, 0, 9), (70, 0, 70)]
EPILOGUES = [  # act, bias, residual, dropout, keep z
    ("none", False, False, None, False),
    ("gelu", True, False, None, True),
    ("silu", True, True, (0.1, 77, 3 << 40), False),
    ("gelu_tanh", False, True, (0.5, (1 << 63) + 5, 1), True),
    ("relu", True, True, None, False),
]


def run_linear(oz, x, w, act, bias, residual, drop, keep, **kw):
    d = {} if drop is None else dict(dropout=drop[0], seed=drop[1], offset=drop[2])
    return oz.linear(x, w, bias=bias, activation=act, residual=residual, return_z=keep, **d, **kw)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
def test_linear(oz, shape, dtype):
    p, q, r = shape
    for k, (act, bias, residual, drop, keep) in enumerate(EPILOGUES):
        pad, shift = [(0, 0), (8, 8), (3, 1), (5, 0), (16, 0)][k]
        print("linear", shape, dtype, act, pad, shift, flush=True)
        x = normal(p, q, dtype, 1 + k, pad=pad, shift=shift)
        w = normal(r, q, dtype, 20 + k, scale=max(q, 1) ** -0.5, pad=pad, shift=shift)
        b = vector(r, dtype, 40 + k) if bias else None
        res = normal(p, r, dtype, 60 + k, pad=pad) if residual else None
        got = run_linear(oz, x, w, act, b, res, drop, keep)
        y, z, ey, ez = ref.linear(x, w, b, act, res, drop)
        ref.assert_within(got[0] if keep else got, y, ey, f"y {act}")
        if keep:
            ref.assert_within(got[1], z, ez, f"z {act}")


@pytest.mark.parametrize("shape", [(2048, 1024, 2304), (1024, 4096, 1024), (4100, 320, 2056), (640, 8200, 520)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
def test_linear_large(oz, shape, dtype):
    """Grids of many tiles, with and without rows on 16-byte boundaries, several depth blocks."""
    p, q, r = shape
    for pad in (0, 1):
        print("linear_large", shape, dtype, pad, flush=True)
        x, w = normal(p, q, dtype, 3, pad=pad), normal(r, q, dtype, 4, scale=q ** -0.5, pad=pad)
        b, res = vector(r, dtype, 5), normal(p, r, dtype, 6)
        got, zg = run_linear(oz, x, w, "gelu", b, res, (0.1, 5, 6), True)
        y, z, ey, ez = ref.linear(x, w, b, "gelu", res, (0.1, 5, 6))
        ref.assert_within(got, y, ey, "y")
        ref.assert_within(zg, z, ez, "z")


@pytest.mark.parametrize("shape", SHAPES + [(1200, 1024, 520), (2048, 2048, 1024), (0, 16, 8), (5, 16, 0)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
def test_linear_backward(oz, shape, dtype):
    p, q, r = shape
    for k, (act, drop) in enumerate([("none", None), ("gelu", (0.1, 9, 8)), ("relu", None), ("gelu_tanh", None),
                                     ("silu", (0.25, 1 << 40, 2)), ("none", (0.5, 1, 1))]):
        pad, shift = [(0, 0), (8, 0), (1, 3), (0, 0), (5, 1), (16, 0)][k]
        print("linear_backward", shape, dtype, act, pad, flush=True)
        dy, x = normal(p, r, dtype, 1 + k, pad=pad, shift=shift), normal(p, q, dtype, 20 + k, pad=pad, shift=shift)
        w = normal(r, q, dtype, 40 + k, scale=max(q, 1) ** -0.5, pad=pad)
        z = normal(p, r, dtype, 60 + k, pad=pad) if act != "none" else None
        d = {} if drop is None else dict(dropout=drop[0], seed=drop[1], offset=drop[2])
        got = oz.linear_backward(dy, x, w, z=z, activation=act, **d)
        want, bound = ref.linear_backward(dy, x, w, z, act, drop)
        for name, g, v, e in zip(("dx", "dw", "db"), got, want, bound):
            ref.assert_within(g, v, e, f"{name} {act}")


def test_linear_backward_of_some(oz):
    """Only what is asked for is computed, and comes out as it does with the rest."""
    dy, x, w, z = normal(70, 90, F16, 1), normal(70, 33, F16, 2), normal(90, 33, F16, 3), normal(70, 90, F16, 4)
    full = oz.linear_backward(dy, x, w, z=z, activation="gelu")
    for needs in [("x",), ("w",), ("bias",), ("x", "bias"), ()]:
        part = oz.linear_backward(dy, x, w, z=z, activation="gelu", needs=needs)
        for name, a, b in zip(("x", "w", "bias"), full, part):
            assert torch.equal(a, b) if name in needs else b is None


@pytest.mark.parametrize("act", ref.ACTS)
def test_gradients_against_differences(oz, act):
    """The kernels' gradients along random directions against central differences of the
    64-bit layer.  Each gradient element is within its bound, so the sum along a direction is
    within the sum of the bounds."""
    dt, drop, (p, q, r) = F16, (0.2, 31, 32), (40, 72, 56)
    x, w, b, dy = normal(p, q, dt, 1), normal(r, q, dt, 2, 0.3), vector(r, dt, 3), normal(p, r, dt, 4)
    _, z = run_linear(oz, x, w, act, b, None, drop, True)
    got = oz.linear_backward(dy, x, w, z=z, activation=act, dropout=drop[0], seed=drop[1], offset=drop[2])
    _, bound = ref.linear_backward(dy, x, w, z, act, drop)
    args = [t.double() for t in (x, w, b)]
    # z is the rounded pre-activation: the 64-bit layer is shifted onto it, so that both take
    # their slopes at the same points
    shift = z.double() - (args[0] @ args[1].t() + args[2])

    def loss(x, w, b):
        return (ref.dropped(ref.activate(x @ w.t() + b + shift, act), drop)[0] * dy.double()).sum()

    g = torch.Generator(device="cuda").manual_seed(9)
    for k in range(3):
        step = torch.randn(args[k].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-7
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + h * step, args[k] - h * step
        diff = (loss(*up) - loss(*down)) / (2 * h)
        # rounding of the two losses (2^-52 of the sums of magnitudes) over 2h, and relu's
        # kinks, which no element sits within h of
        noise = 2.0 ** -50 * dy.double().abs().sum() * 20 / h + 1e-5
        assert abs(diff - (got[k].double() * step).sum()) <= (bound[k] * step.abs()).sum() + noise, (act, k)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (3, 8), (5, 9), (16, 2048), (1000, 63), (257, 2049), (70000, 5)], ids=str)
def test_dropout_add(oz, dtype, shape):
    p, r = shape
    for prob, seed, offset, pad, with_res in [(0.1, 3, 4, 0, True), (0.5, (1 << 64) - 1, (1 << 64) - 1, 3, False),
                                              (0.0, 0, 0, 1, True), (1.0, 5, 6, 0, True), (1e-9, 7, 7, 8, True)]:
        print("dropout_add", dtype, shape, prob, flush=True)
        x = normal(p, r, dtype, 1, pad=pad, shift=pad % 2)
        res = normal(p, r, dtype, 2, pad=pad) if with_res else None
        got = oz.dropout_add(x, res, dropout=prob, seed=seed, offset=offset)
        want, scale = ref.dropped(x.double(), (prob, seed, offset))
        # f32 arithmetic: the scale, the product and the sum round once each
        bound = 2 * 2.0 ** -24 * want.abs()
        if with_res:
            want = want + res.double()
        ref.assert_within(got, want, (bound + ref.rounding(want, dtype)) * 1.01 + (2.0 ** -24 * want.abs()), f"{prob}")
        keep, _ = ref.keep_and_scale(p, r, (prob, seed, offset), "cuda")
        if not with_res:
            assert torch.equal(got != 0, keep & (x != 0))
            # the gradient is the same call on dy
            dx = oz.dropout_add(torch.ones_like(x), dropout=prob, seed=seed, offset=offset)
            assert torch.equal(dx != 0, keep)


def test_dropped_elements_are_zero_whatever_they_hold(oz):
    p, r, drop = 64, 96, (0.5, 8, 9)
    keep, scale = ref.keep_and_scale(p, r, drop, "cuda")
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = torch.where(keep, 1.0, bad).to(BF16)
        assert torch.equal(oz.dropout_add(x, dropout=drop[0], seed=drop[1], offset=drop[2]),
                           (keep * scale).to(BF16))
        # in the epilogue: a bias that makes whole columns non-finite reaches kept elements only
        bias = torch.zeros(r, dtype=BF16, device="cuda")
        bias[5] = bad
        y = oz.linear(torch.zeros(p, 16, dtype=BF16, device="cuda"), torch.zeros(r, 16, dtype=BF16, device="cuda"),
                      bias=bias, residual=torch.ones(p, r, dtype=BF16, device="cuda"), dropout=drop[0], seed=drop[1],
                      offset=drop[2])
        assert torch.equal(torch.isfinite(y[:, 5]), ~keep[:, 5]) and torch.isfinite(y[:, :5]).all()
        # in the gradient: dY's non-finite dropped elements reach nothing
        dy = torch.where(keep, 1.0, bad).to(BF16)
        for g in oz.linear_backward(dy, torch.ones(p, 24, dtype=BF16, device="cuda"),
                                    torch.ones(r, 24, dtype=BF16, device="cuda"), dropout=drop[0], seed=drop[1],
                                    offset=drop[2]):
            assert torch.isfinite(g).all()


@pytest.mark.parametrize("act", ref.ACTS)
def test_non_finite_rows_stay_in_their_rows(oz, act):
    """Inf and NaN of one token reach that token's outputs as the formula says, and no other's."""
    for p, q, r in [(5, 64, 40), (300, 96, 200)]:
        x, w = normal(p, q, F16, 1), normal(r, q, F16, 2)
        x[1, 3], x[2, 5] = float("inf"), float("nan")
        y, _ = run_linear(oz, x, w, act, None, None, None, True)
        want, _, bound, _ = ref.linear(x, w, None, act)
        clean = torch.ones(p, dtype=torch.bool, device="cuda")
        clean[1:3] = False
        ref.assert_within(y[clean], want[clean], bound[clean], act)
        assert torch.isnan(y[2]).all()
        assert torch.equal(torch.isnan(y[1]), torch.isnan(want[1])), act


@pytest.mark.parametrize("act", ref.ACTS)
def test_activations_over_their_range(oz, act):
    """Bias alone sets the pre-activation: the whole range of the type, tails and both zeros."""
    for dtype in (BF16, F16):
        a = torch.cat([torch.linspace(-30, 30, 4001), torch.tensor([0.0, -0.0, 1e-7, -1e-7, 6e4, -6e4])]).to(dtype).cuda()
        n = a.numel()
        y = oz.linear(torch.zeros(1, 8, dtype=dtype, device="cuda"), torch.zeros(n, 8, dtype=dtype, device="cuda"),
                      bias=a, activation=act)
        want = ref.activate(a.double(), act)[None]
        # relative 2^-20 of |a| + 1 beside the rounding
        ref.assert_within(y, want, ref.rounding(want, dtype) + 2.0 ** -20 * (1 + a.double().abs()).clamp(max=64), act)
        # slopes, through the gradient of a layer whose W is the identity
        g = oz.linear_backward(torch.ones(1, n, dtype=dtype, device="cuda"), torch.zeros(1, 1, dtype=dtype, device="cuda"),
                               torch.zeros(n, 1, dtype=dtype, device="cuda"), z=a[None], activation=act, needs=("bias",))[2]
        ds = ref.slope(a.double(), act)
        ref.assert_within(g, ds, ref.rounding(ds, dtype) + 2.0 ** -19, act)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 17), (40, 256), (7, 2049), (300, 8192), (2, 20000), (4, 0)], ids=str)
def test_quantize_rows(oz, dtype, shape):
    for pad in (0, 3):
        x = normal(*shape, dtype, 1, pad=pad, shift=pad)
        if shape[0] > 2 and shape[1] > 5:
            x[0] = 0
            x[1, 2], x[2, 5] = float("inf"), float("nan")
        q, s = oz.quantize_rows(x)
        wq, ws = ref.quantize(x)
        assert torch.equal(q, wq)
        assert torch.equal(torch.nan_to_num(s, nan=-1.0), torch.nan_to_num(ws, nan=-1.0))


def test_quantize_tiny_rows(oz):
    x = torch.tensor([[1e-37, -3e-38, 0.0], [2e-36, -1e-36, 1e-40], [3e38, -1e38, 1.0]], device="cuda")
    q, s = oz.quantize_rows(x)
    wq, ws = ref.quantize(x)
    assert torch.equal(q, wq) and torch.equal(s, ws)


@pytest.mark.parametrize("shape", SHAPES + [(2048, 1024, 2304), (640, 8200, 520), (37, 131072, 16)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
def test_linear_i8(oz, shape, dtype):
    p, q, r = shape
    for k, (act, bias, residual, _, _) in enumerate(EPILOGUES):
        pad = [0, 16, 3, 0, 5][k]
        print("linear_i8", shape, dtype, act, pad, flush=True)
        x, w = normal(p, q, dtype, 1 + k, pad=pad), normal(r, q, dtype, 20 + k, scale=max(q, 1) ** -0.5)
        v, t = oz.quantize_rows(w)
        if pad:
            wide = torch.zeros(r, q + pad, dtype=torch.int8, device="cuda")
            wide[:, :q] = v
            v = wide[:, :q]
        b = vector(r, dtype, 40 + k) if bias else None
        res = normal(p, r, dtype, 60 + k) if residual else None
        got = oz.linear_i8(x, v, t, bias=b, activation=act, residual=res)
        want, bound = ref.linear_i8(x, v, t, b, act, res)
        ref.assert_within(got, want, bound, act)


def test_linear_i8_extremes_are_exact(oz):
    """Levels of +-127 throughout: the largest int32 sums, 127^2 131072, exact."""
    q = 131072
    for p in (2, 200):
        x = torch.ones(p, q, dtype=F16, device="cuda")
        x[1] = -1
        v = torch.full((72, q), 127, dtype=torch.int8, device="cuda")
        v[1] = -127
        t = torch.full((72,), 2.0 ** -24, device="cuda")
        want, bound = ref.linear_i8(x, v, t)
        ref.assert_within(oz.linear_i8(x, v, t), want, bound, "extremes")


def test_linear_i8_non_finite_rows(oz):
    for p in (4, 150):
        x, w = normal(p, 64, F16, 1), normal(70, 64, F16, 2)
        x[1, 3], x[2, 5], x[3] = float("inf"), float("nan"), 0
        v, t = oz.quantize_rows(w)
        want, bound = ref.linear_i8(x, v, t)
        got = oz.linear_i8(x, v, t)
        assert torch.isnan(got[1:3]).all()
        ref.assert_within(got[3:], want[3:], bound[3:], "rows")
        ref.assert_within(got[:1], want[:1], bound[:1], "rows")


def test_output_in_place_of_residual_and_in_wide_buffers(oz):
    for p, q, r in [(4, 64, 48), (200, 128, 136)]:
        for dtype in (BF16, F16):
            x, w, res = normal(p, q, dtype, 1), normal(r, q, dtype, 2, 0.1), normal(p, r, dtype, 3)
            want = oz.linear(x, w, residual=res, activation="silu")
            # input, residual and output as column ranges of one buffer; what lies between stays
            wide = torch.full((p, q + 2 * r + 8), 7.0, dtype=dtype, device="cuda")
            wide[:, :q], wide[:, q:q + r] = x, res
            out = wide[:, q + r + 3:q + 2 * r + 3]
            got = oz.linear(wide[:, :q], w, residual=wide[:, q:q + r], activation="silu", out=out)
            assert torch.equal(got, want) and got.data_ptr() == out.data_ptr()
            assert torch.equal(wide[:, :q], x) and torch.equal(wide[:, q:q + r], res)
            assert (wide[:, q + r:q + r + 3] == 7).all() and (wide[:, q + 2 * r + 3:] == 7).all()
            inplace = res.clone()
            assert torch.equal(oz.linear(x, w, residual=inplace, activation="silu", out=inplace), want)
            d = oz.dropout_add(res, x[:, :1].expand(p, r).contiguous(), dropout=0.3, seed=1)
            same = res.clone()
            oz.dropout_add(same, x[:, :1].expand(p, r).contiguous(), dropout=0.3, seed=1, out=same)
            assert torch.equal(same, d)


def test_rows_beyond_32_bit_offsets(oz):
    """Element offsets past 2^31 (and byte offsets past 2^32): a few columns of a wide buffer."""
    p, wide = 70001, 32768
    buf = torch.empty(p, wide, dtype=F16, device="cuda")
    x = buf[:, 100:124]
    x.copy_(normal(p, 24, F16, 1))
    got = oz.dropout_add(x, None, dropout=0.5, seed=1, offset=2, out=buf[:, 1000:1024])
    want, scale = ref.dropped(x[-9:].double(), None)
    keep = torch.from_numpy(ref.draws(9, 24, 1, 2, row0=p - 9) >= 32768).cuda()
    assert torch.equal(got[-9:].double(), torch.where(keep, want * 2, 0.0))
    w = normal(40, 24, F16, 2)
    y = oz.linear(x, w, out=buf[:, 2000:2040])
    yw, _, bound, _ = ref.linear(x[-300:], w)
    ref.assert_within(y[-300:], yw, bound, "tail rows")
    dy = buf[:, 2000:2040]
    dx, dw, db = oz.linear_backward(dy, x, w)
    want, bound = ref.linear_backward(dy, x, w)
    for name, g, v, e in zip(("dx", "dw", "db"), (dx, dw, db), want, bound):
        ref.assert_within(g, v, e, name)


def test_repeats_give_the_same_bits(oz):
    x, w, dy, z = normal(500, 1000, BF16, 1), normal(700, 1000, BF16, 2), normal(500, 700, BF16, 3), normal(500, 700, BF16, 4)
    few = normal(3, 1000, BF16, 5)
    v, t = oz.quantize_rows(w)
    first = None
    for _ in range(3):
        out = [oz.linear(x, w, activation="gelu", dropout=0.1, seed=1), oz.linear(few, w), oz.linear_i8(few, v, t),
               *oz.linear_backward(dy, x, w, z=z, activation="gelu")]
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_streams_and_library_workspace(oz):
    """Calls on two streams at once give what they give alone; without a caller's scratch the
    library's own buffer serves, is freed by ozaki2_release, and comes back."""
    x, w, dy, z = normal(300, 256, F16, 1), normal(400, 256, F16, 2, 0.1), normal(300, 400, F16, 3), normal(300, 400, F16, 4)
    want = oz.linear_backward(dy, x, w, z=z, activation="gelu", dropout=0.1, seed=4)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [oz.linear_backward(dy, x, w, z=z, activation="gelu", dropout=0.1, seed=4, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    dx, dw, db = (torch.empty_like(t) for t in want)
    for _ in range(2):
        rc = oz.ozaki2_linear_bwd(oz.OZ2_F16, 300, 256, 400, dy.data_ptr(), 400, x.data_ptr(), 256, w.data_ptr(), 256,
                                  z.data_ptr(), 400, oz.OZ2_ACT_GELU, oz.OZ2Dropout(0.1, 4, 0), dx.data_ptr(), 256,
                                  dw.data_ptr(), 256, db.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
        assert rc == oz.OZ2_OK
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), want))
        assert oz.ozaki2_release() == oz.OZ2_OK


def test_flags_of_a_product_survive_linear_calls(oz):
    """The FP64 product's flag word stays readable after linear-layer calls, on the library's
    workspaces and on a shared caller workspace."""
    a = oz.colmajor(torch.randn(64, 64, dtype=torch.float64, device="cuda"))
    a[3, 3] = float("inf")
    x, w = normal(64, 64, F16, 1), normal(64, 64, F16, 2)
    v, t = oz.quantize_rows(w)
    buf = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def i8():
        y = torch.empty(64, 64, dtype=F16, device="cuda")
        rc = oz.ozaki2_linear_i8(oz.OZ2_F16, 64, 64, 64, x.data_ptr(), 64, v.data_ptr(), 64, t.data_ptr(), None,
                                 oz.OZ2_ACT_NONE, None, 64, y.data_ptr(), 64, None, 0, torch.cuda.current_stream().cuda_stream)
        assert rc == oz.OZ2_OK
        return y

    want = oz.linear_i8(x, v, t)
    for set_ws in (False, True):
        assert oz.ozaki2_set_workspace(buf.data_ptr() if set_ws else None, buf.numel() if set_ws else 0) == oz.OZ2_OK
        try:
            oz.dgemm(a, a, s=8)
            assert torch.equal(i8(), want)
            assert oz.ozaki2_get_flags() == (oz.OZ2_OK, oz.OZ2_FLAG_NONFINITE)
        finally:
            assert oz.ozaki2_set_workspace(None, 0) == oz.OZ2_OK


def test_graph_replays(oz):
    """A captured training step and a captured single-token step, replayed with eager work and
    synchronisations between, each replay checked against the eager result on new inputs."""
    for p in (1, 260):
        x, w, b = normal(p, 512, BF16, 1), normal(384, 512, BF16, 2, 0.05), vector(384, BF16, 3)
        dy = normal(p, 384, BF16, 4)
        v, t = oz.quantize_rows(w)

        def step():
            y, z = oz.linear(x, w, bias=b, activation="gelu", dropout=0.1, seed=3, return_z=True)
            g = oz.linear_backward(dy, x, w, z=z, activation="gelu", dropout=0.1, seed=3)
            return [y, z, *g, oz.linear_i8(x, v, t, bias=b), oz.dropout_add(y, z, dropout=0.5, seed=2)]

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for k in range(4):
            x.copy_(normal(p, 512, BF16, 100 + k))
            dy.copy_(normal(p, 384, BF16, 200 + k))
            want = [t.clone() for t in step()]
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), k


def test_refusals_of_device_tensors(oz):
    x, w = normal(8, 16, BF16, 1), normal(12, 16, BF16, 2)
    with pytest.raises(ValueError, match="row-major"):
        oz.linear(x, normal(16, 12, BF16, 2).t())
    with pytest.raises(ValueError, match="row-major"):
        oz.linear(x[:1].expand(8, 16), w)
    with pytest.raises(ValueError, match="shape"):
        oz.linear(x, w, residual=normal(1, 12, BF16, 3))
    with pytest.raises(ValueError, match="shape"):
        oz.linear(x, w, bias=vector(11, BF16, 3))
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        oz.linear(x, w.half())
    with pytest.raises(ValueError, match="contiguous"):
        oz.linear(x, w, bias=normal(12, 2, BF16, 3)[:, 0])
    with pytest.raises(ValueError, match="device"):
        oz.linear(x, w.cpu())
    with pytest.raises(oz.Oz2Error):
        oz.linear(x, w, out=x[:, :12])
    with pytest.raises(ValueError, match="torch.int8"):
        oz.linear_i8(x, w, torch.ones(12, device="cuda"))
    with pytest.raises(ValueError, match="torch.float32"):
        oz.linear_i8(x, w.to(torch.int8), vector(12, BF16, 1))
