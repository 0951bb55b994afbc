"""Views that start off a 16-byte border give what aligned tensors give."""
import pytest
import torch

from clustering_flashassign_b200.soft import expert_mixture, token_log_probs

pytestmark = pytest.mark.gpu


def off_border(t):
    """The same values in a contiguous tensor that starts 2 or 4 bytes off a 16-byte border."""
    room = torch.empty(t.numel() + 1, device=t.device, dtype=t.dtype)
    v = room[1:].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16
    return v


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_views_off_a_16_byte_border(dtype):
    x = torch.randn(30, 24, device="cuda").to(dtype)
    c = torch.randn(50, 24, device="cuda").to(dtype)
    b = torch.randn(50, device="cuda")
    ids = torch.randint(0, 50, (30,), device="cuda", dtype=torch.int32)

    def both(x, c, b, ids):
        leaves = [x.detach().requires_grad_(True), c.detach().requires_grad_(True), b.detach().requires_grad_(True)]
        r = token_log_probs(leaves[0], leaves[1], ids, bias=leaves[2], top=3)
        return [*r, *torch.autograd.grad([r.logp.sum() + r.entropy.sum()], leaves)]

    want = both(x, c, b, ids)
    got = both(off_border(x), off_border(c), off_border(b), off_border(ids))
    assert all(torch.equal(u, v) for u, v in zip(want, got))
    if dtype != torch.float32:
        moe = [(torch.randn(*s, device="cuda") / 4).to(dtype) for s in ((6, 24), (5, 24), (5, 32, 24), (5, 24, 16))]
        assert all(torch.equal(u, v) for u, v in zip(expert_mixture(*moe, 2),
                                                     expert_mixture(*[off_border(t) for t in moe], 2)))
