"""Alternatives of a table whose scores lie closer than fp32 tells apart.

What is returned is ordered by the fp64 scores, and every returned column's score is
within twice the fp32 score's error (score_tol of test_logprob.py) of the place it takes.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [7, 5000])
@pytest.mark.parametrize("top", [1, 5, 20])
def test_near_duplicates_of_one_row(N, top):
    from clustering_flashassign_b200.soft import token_log_probs
    from test_logprob import reference, score_tol
    K, d = 300, 96
    g = torch.Generator(device="cuda").manual_seed(top)
    row = torch.randn(1, 1, d, generator=g, device="cuda")
    c = row + 1e-6 * torch.randn(1, K, d, generator=g, device="cuda")
    x = torch.randn(1, N, d, generator=g, device="cuda")
    ids = torch.zeros(1, N, device="cuda", dtype=torch.int32)
    r = token_log_probs(x, c, ids, top=top)
    s, lp, p, lse, logp, ent, A = reference(x, c, ids, 1.0, None)
    tol = score_tol(x, A, s).unsqueeze(-1)
    got = s.gather(-1, r.top_ids.long())
    assert (got[..., 1:] <= got[..., :-1] + 2.0 ** -48 * s.abs().amax()).all()
    assert (got >= s.sort(-1, descending=True).values[..., :top] - 2 * tol).all()
    ordered = r.top_ids.sort(-1).values
    assert (ordered[..., 1:] > ordered[..., :-1]).all()  # no column twice
