"""The linear-layer functions beside autograd: what would lose a gradient is refused (before any
library call, so on the CPU), what runs is known to autograd as written."""
import pytest
import torch

from fp64_gemm_emulation_amd import binding as oz


SIZES = {"linear": dict(x=(4, 16), w=(8, 16), bias=(8,), residual=(4, 8), out=(4, 8)),
         "dropout_add": dict(x=(4, 8), residual=(4, 8), out=(4, 8)),
         "linear_i8": dict(x=(4, 16), t=(8,), bias=(8,), residual=(4, 8), out=(4, 8))}


def operands(name, grad=None, device="cpu"):
    t = {k: torch.zeros(*s, dtype=torch.float32 if k == "t" else torch.float16, device=device).requires_grad_(k == grad)
         for k, s in SIZES[name].items()}
    if name == "linear_i8":
        t["v"] = torch.zeros(8, 16, dtype=torch.int8, device=device)
    return t


@pytest.mark.parametrize("name, operand", [(n, o) for n in SIZES for o in SIZES[n]])
def test_a_lost_gradient_is_refused(name, operand):
    with pytest.raises(ValueError, match="autograd"):
        getattr(oz, name)(**operands(name, operand))
    # with gradients off the call goes on (to its refusal of host tensors)
    for off in (torch.no_grad, torch.inference_mode):
        with off(), pytest.raises(ValueError, match="CUDA"):
            getattr(oz, name)(**operands(name, operand))
    with pytest.raises(ValueError, match="CUDA"):
        getattr(oz, name)(**operands(name))


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(SIZES))
def test_a_written_tensor_has_a_new_version(name):
    t = operands(name, device="cuda")
    scale = torch.ones(4, 8, dtype=torch.float16, device="cuda", requires_grad=True)
    loss = (t["out"] * scale).sum()          # saves out for scale's gradient
    before = t["out"]._version
    assert getattr(oz, name)(**t) is t["out"] and t["out"]._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.gpu
def test_parameters_with_gradients_off():
    """Parameters and tensors of inference mode as operands and outputs."""
    t = operands("linear", device="cuda")
    want = oz.linear(**t)
    t["w"] = torch.nn.Parameter(t["w"])
    with torch.no_grad():
        assert torch.equal(oz.linear(**t), want)
    with torch.inference_mode():
        t["out"] = torch.empty(4, 8, dtype=torch.float16, device="cuda")
        assert torch.equal(oz.linear(**t), want)
