"""Upstream gradients that overflowed (a scaled loss) stay the business of their own rows."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(50, 3000), (700, 9000)])
def test_other_rows_keep_their_gradients(N, K, dtype, bad):
    from clustering_flashassign_b200.soft import token_log_probs
    from test_logprob import make
    x, c, ids, _ = make(1, N, K, 64, dtype, seed=N, ignore=0.0)
    up = torch.randn(1, N, device="cuda")
    up[0, 7] = 0.0
    broken = up.clone()
    broken[0, 7] = bad

    def dx(u):
        leaf = x.clone().requires_grad_(True)
        return torch.autograd.grad([token_log_probs(leaf, c, ids).logp], leaf, [u])[0]

    want, got = dx(up), dx(broken)
    rows = torch.arange(N, device="cuda") != 7
    assert torch.equal(want[0, rows], got[0, rows])
    assert not torch.isfinite(got[0, 7]).any()
