"""The feed-forward example: the operators together, trained and served."""
import importlib.util
import os

import pytest

from tests import linear_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_trains_and_serves(example):
    out = example.run(tokens=512, width=256, hidden=1024, steps=30)
    losses = out["losses"]
    assert all(v == v for v in losses) and losses[-1] < 0.8 * losses[0], losses
    # the stream's value, of order 1, is rounded to 2^-8 of itself beside an addition of like size
    assert out["bf16"] < 0.02
    # row scales: levels of 1/127 of a row's largest, about 1% of a typical element each
    assert out["int8"] < 0.05


def test_gradients_of_the_block(example):
    """The block's gradients against autograd of its 64-bit form on the same rounded weights and
    masks.  Every tensor is rounded to bfloat16 between the operators (2^-9 of it, root mean
    square below that), a handful of times in a row: 2% in norm is several times their sum."""
    block = example.FeedForward(96, 200, 0.2, seed=3)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, pos, dy = (torch.randn(70, 96, generator=g, device="cuda").bfloat16() for _ in range(3))
    _, saved = block.forward(x, pos, 5)
    grads, dx, dpos = block.backward(dy, saved, 5)
    leaves = {k: getattr(block, k).double().requires_grad_() for k in ("w1", "b1", "w2", "b2")}
    xt, pt = x.double().requires_grad_(), pos.double().requires_grad_()
    masks = []
    for place, cols in ((0, 96), (1, 96)):
        d = block.drop(5, place)
        keep, scale = ref.keep_and_scale(70, cols, (d["dropout"], d["seed"], d["offset"]), "cuda")
        masks.append(keep.double() * scale)
    s = xt + pt * masks[0]
    a = s @ leaves["w1"].t() + leaves["b1"]
    y = s + (ref.activate(a, "gelu") @ leaves["w2"].t() + leaves["b2"]) * masks[1]
    y.backward(dy.double())
    for name, got, want in [(k, grads[k], leaves[k].grad) for k in leaves] + [("x", dx, xt.grad), ("pos", dpos, pt.grad)]:
        assert (got.double() - want).norm() <= 0.02 * want.norm(), name
