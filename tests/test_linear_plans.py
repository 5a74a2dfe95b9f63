"""Which kernel the sizes of the kernel tests run on, without a GPU: a rule or a constant that
moves one of them elsewhere fails here."""
import pytest

from tests import linear_plans as plans


@pytest.mark.parametrize("shape, tile, split", plans.FORWARD, ids=str)
def test_forward(shape, tile, split):
    assert plans.kernel(plans.forward(*shape)) == (tile, split)


@pytest.mark.parametrize("shape, tile, split", plans.INT8, ids=str)
def test_int8(shape, tile, split):
    assert plans.kernel(plans.int8(*shape)) == (tile, split)


@pytest.mark.parametrize("shape, paired, dx, dw", plans.BACKWARD, ids=str)
def test_backward(shape, paired, dx, dw):
    got = plans.backward(*shape)
    assert (got[0], plans.kernel(got[1]), plans.kernel(got[2])) == (paired, dx, dw)


def test_every_kernel_has_sizes():
    """All kernels, split where they can be, in every direction they serve."""
    tiles = {(t, s) for t in ("tile128", "tile128deep", "tile64") for s in (False, True)} | {("tile256", False)}
    few = {("few8", False), ("few16", False)}
    assert {(t, s) for _, t, s in plans.FORWARD} == tiles | few
    assert {(t, s) for _, t, s in plans.INT8} == tiles | few
    assert {dx for _, paired, dx, _ in plans.BACKWARD if not paired} == tiles
    # dW's left operand lies along its index, which 64-row tiles do not take
    assert {dw for _, paired, _, dw in plans.BACKWARD if not paired} == {t for t in tiles if t[0] != "tile64"}
    assert {(dx, dw) for _, paired, dx, dw in plans.BACKWARD if paired} >= {
        (("tile128deep", True), ("tile128deep", False)), (("tile128deep", False), ("tile128deep", True)),
        (("tile128deep", False), ("tile128deep", False))}
