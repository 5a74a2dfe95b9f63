"""The gradients of norm and log probabilities have no gradients of their own: operands for which
autograd would be asked for one are refused, as the forward calls refuse theirs."""
import pytest
import torch

from fp64_gemm_emulation_amd import binding as oz

CALLS = {
    "rms_norm_backward": dict(dy=(4, 16), h=(4, 16), weight=(16,), dh=(4, 16)),
    "token_logprobs_backward": dict(dlogprobs=(4,), logits=(4, 16), lse=(4,), dentropy=(4,), entropy=(4,), out=(4, 16)),
}


@pytest.mark.parametrize("name, operand", [(n, o) for n, sizes in CALLS.items() for o in sizes])
def test_a_lost_gradient_is_refused(name, operand):
    t = {k: torch.zeros(s).requires_grad_(k == operand) for k, s in CALLS[name].items()}
    if name == "token_logprobs_backward":
        t["tokens"] = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="autograd"):
        getattr(oz, name)(**t)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        getattr(oz, name)(**t)
