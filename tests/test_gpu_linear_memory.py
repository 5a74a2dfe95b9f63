"""Memory that linear-layer calls leave in use: the library's own buffer under a captured graph,
operands and outputs of calls on another stream."""
import pytest

from tests.test_gpu_linear import F16, normal, oz, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def test_graph_on_the_librarys_buffer_outlives_larger_calls(oz):  # noqa: F811
    """A call captured without a caller's scratch, replayed after larger calls have made the
    library take another buffer, with eager work and new allocations between the replays."""
    def operands(p, q, r, seed):
        return normal(p, r, F16, seed), normal(p, q, F16, seed + 1), normal(r, q, F16, seed + 2, 0.1), normal(p, r, F16, seed + 3)

    def backward(dy, x, w, z, dx, dw, db):
        (p, r), q = dy.shape, x.shape[1]
        rc = oz.ozaki2_linear_bwd(oz.OZ2_F16, p, q, r, dy.data_ptr(), r, x.data_ptr(), q, w.data_ptr(), q, z.data_ptr(), r,
                                  oz.OZ2_ACT_GELU, None, dx.data_ptr(), q, dw.data_ptr(), q, db.data_ptr(), None, 0,
                                  torch.cuda.current_stream().cuda_stream)
        assert rc == oz.OZ2_OK

    assert oz.ozaki2_release() == oz.OZ2_OK
    small = operands(256, 256, 1024, 1)
    out = [torch.empty(s, dtype=F16, device="cuda") for s in ((256, 256), (1024, 256), (1024,))]
    backward(*small, *out)  # the library's buffer has its size
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        backward(*small, *out)
    for k, n in enumerate((512, 1024, 2048)):
        large = operands(n, n, n, 10 + k)
        grads = [torch.empty(s, dtype=F16, device="cuda") for s in ((n, n), (n, n), (n,))]
        backward(*large, *grads)
        want = oz.linear_backward(*large[:3], z=large[3], activation="gelu")
        assert all(torch.equal(a, b) for a, b in zip(grads, want))
        small[0].copy_(normal(256, 1024, F16, 30 + k))
        want = oz.linear_backward(*small[:3], z=small[3], activation="gelu")
        filled = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and (filled == 0xFF).all()
    del graph
    assert oz.ozaki2_release() == oz.OZ2_OK


CALLS = {  # operands by their sizes, and the call on them
    "linear": (dict(x=(700, 512), w=(600, 512), bias=(600,), residual=(700, 600)), lambda oz, t, **kw: oz.linear(**t, **kw)),
    "backward": (dict(dy=(700, 600), x=(700, 512), w=(600, 512), z=(700, 600)),
                 lambda oz, t, **kw: oz.linear_backward(**t, activation="gelu", **kw)),
    "dropout_add": (dict(x=(1000, 801), residual=(1000, 801)), lambda oz, t, **kw: oz.dropout_add(**t, dropout=0.5, **kw)),
    "quantize_rows": (dict(x=(900, 700)), lambda oz, t, **kw: oz.quantize_rows(**t, **kw)),
    "linear_i8": (dict(x=(700, 512), v=(600, 512), t=(600,), bias=(600,), residual=(700, 600)),
                  lambda oz, t, **kw: oz.linear_i8(**t, **kw)),
}


def make(sizes):
    torch.manual_seed(1)
    t = {k: (torch.randn(s, device="cuda") * 0.1).half() for k, s in sizes.items()}
    if "v" in t:
        t["v"], t["t"] = (t["v"] * 100).to(torch.int8), t["t"].float().abs()
    return t


@pytest.mark.parametrize("name", list(CALLS))
def test_operands_dropped_after_a_call_on_a_stream(oz, name):  # noqa: F811
    """stream= reads the operands later than the caller lets go of them: their memory stays theirs
    until the call is done, though the caller's stream has been given new tensors meanwhile."""
    sizes, call = CALLS[name]
    plain = call(oz, make(sizes))
    want = [t.clone() for t in (plain if isinstance(plain, tuple) else (plain,))]
    # what a tensor without another stream's use does: its memory comes back at once
    a = torch.empty(5 << 20, dtype=torch.uint8, device="cuda")
    at = a.data_ptr()
    del a
    a = torch.empty(5 << 20, dtype=torch.uint8, device="cuda")
    assert a.data_ptr() == at
    s = torch.cuda.Stream()
    busy = torch.randn(8192, 8192, device="cuda")
    torch.mm(busy, busy)
    operands = make(sizes)
    places = {t.data_ptr() for t in operands.values()}
    shapes = [(t.shape, t.dtype) for t in operands.values()]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(8):
            torch.mm(busy, busy)
    got = call(oz, operands, stream=s)
    del operands
    assert not s.query(), "the stream is still busy before the call"
    others = [torch.full(shape, 77, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(2)]
    assert not s.query()
    assert not places & {t.data_ptr() for t in others}
    torch.cuda.synchronize()
    for a, b in zip(got if isinstance(got, tuple) else (got,), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs_dropped_while_the_callers_stream_reads_them(oz, name):  # noqa: F811
    """Outputs made on stream= and used on the caller's stream: let go of there, their memory does
    not go to the next call on stream= before that use is done."""
    sizes, call = CALLS[name]
    s = torch.cuda.Stream()
    operands = make(sizes)
    plain = call(oz, operands)
    want = [t.clone() for t in (plain if isinstance(plain, tuple) else (plain,))]
    busy = torch.randn(8192, 8192, device="cuda")
    torch.mm(busy, busy)
    torch.cuda.synchronize()
    got = call(oz, operands, stream=s)
    got = got if isinstance(got, tuple) else (got,)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(8):
        torch.mm(busy, busy)
    read = [t.clone() for t in got]
    places = {t.data_ptr() for t in got}
    del got
    again = call(oz, operands, stream=s)
    assert not torch.cuda.current_stream().query(), "the reads are still to come"
    assert not places & {t.data_ptr() for t in (again if isinstance(again, tuple) else (again,))}
    torch.cuda.synchronize()
    for a, b in zip(read, want):
        assert torch.equal(a, b)
