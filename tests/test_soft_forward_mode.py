"""Forward-mode derivatives of the soft assignment operators are refused, not dropped."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

from clustering_flashassign_b200.soft import expert_mixture, token_log_probs


def inputs(device):
    def t(*s):
        return torch.randn(*s, device=device).half()

    ids = torch.zeros(4, device=device, dtype=torch.int32)
    return (t(4, 16), t(20, 16), torch.zeros(20, device=device)), ids, (t(4, 16), t(5, 16), t(5, 16, 16), t(5, 16, 8))


def refused(device):
    (x, c, b), ids, moe = inputs(device)
    for grad in (True, False):
        with torch.set_grad_enabled(grad), fwd.dual_level():
            for i in range(3):
                args = [x, c, b]
                args[i] = fwd.make_dual(args[i], torch.ones_like(args[i]))
                with pytest.raises(RuntimeError, match="forward-mode"):
                    token_log_probs(args[0], args[1], ids, bias=args[2])
            for i in range(4):
                args = list(moe)
                args[i] = fwd.make_dual(args[i], torch.ones_like(args[i]))
                with pytest.raises(RuntimeError, match="forward-mode"):
                    expert_mixture(*args, 2)


def test_duals_are_refused_before_anything_else():
    refused("cpu")


@pytest.mark.gpu
def test_duals_are_refused_and_plain_tensors_of_the_level_are_not():
    refused("cuda")
    (x, c, b), ids, moe = inputs("cuda")
    with fwd.dual_level():
        assert torch.isfinite(token_log_probs(x, c, ids, bias=b).logp).all()
        assert torch.isfinite(expert_mixture(*moe, 2).y).all()
        g = torch.autograd.grad(token_log_probs(x.requires_grad_(True), c, ids).logp.sum(), x)[0]
        assert torch.isfinite(g).all()
