"""Scores so large that fp32 holds whole numbers only: a row's sum does not get lost beside them."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def run(x, c, ids, bias, top, up):
    from clustering_flashassign_b200.soft import token_log_probs
    leaves = [t.clone().requires_grad_(True) for t in (x, c, bias)]
    r = token_log_probs(leaves[0], leaves[1], ids, bias=leaves[2], top=top)
    return r, torch.autograd.grad([r.logp, r.lse, r.entropy], leaves, up)


@pytest.mark.parametrize("shift", [0.0, 2.0 ** 20, 2.0 ** 23, 2.0 ** 24, 2.0 ** 27, 1e9, -1e9])
@pytest.mark.parametrize("N,top", [(5, 3), (5, 0), (200, 0), (5000, 3), (5000, 15)])
def test_equal_scores_of_any_size(shift, N, top):
    """x = 0: every column has the bias, and log p = -log K whatever its size."""
    K, d = 700, 40
    x = torch.zeros(1, N, d, device="cuda", dtype=torch.bfloat16)
    c = torch.randn(1, K, d, device="cuda").bfloat16()
    ids = torch.randint(0, K, (1, N), device="cuda", dtype=torch.int32)
    bias = torch.full((1, K), shift, device="cuda")
    up = [torch.ones(1, N, device="cuda"), torch.zeros(1, N, device="cuda"), torch.zeros(1, N, device="cuda")]
    r, (dx, dc, db) = run(x, c, ids, bias, top, up)
    assert ((r.logp + math.log(K)).abs() <= 16 * U * math.log(K)).all()
    assert ((r.entropy - math.log(K)).abs() <= 16 * U * math.log(K)).all()
    if top:
        assert (r.top_ids == torch.arange(top, device="cuda", dtype=torch.int32)).all()
        assert ((r.top_logp + math.log(K)).abs() <= 16 * U * math.log(K)).all()
    count = torch.bincount(ids[0].long(), minlength=K).double()
    want = count - N / K
    # p from lse, held to 2^-47 of its size (at most 3e9 in base 2), and fp32 sums of N terms
    assert ((db[0].double() - want).abs() <= N / K * 2.0 ** -15 + (count + N / K) * (N / 32 + 8) * U).all()
    assert (dc == 0).all()
