"""Memory that linear-layer calls leave in use: the library's own buffer under a captured graph."""
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
