"""Gradients of confident rows over deep contractions: 1 - p of the target is small, so
a gradient is what is left of terms that nearly cancel.

A row's p must be normalised by the lse of the same scores.  Bound per value, against
fp64, for a row with upstream a and score error tol (see test_logprob.py): the other
columns' p are off by 4 tol of themselves, the target's 1 - p by 4 tol of itself and by
the two exponentials (2 ulp each), the sum's joins and its logarithm: 2^-20; G is rounded
by half a step (twice where it is held in two parts); an accumulation over n terms adds
(n / 16 + 20) roundings of 2^-23; the result is rounded by half a step.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -23


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N,K,d", [(40, 300, 2048), (200, 300, 4096), (1100, 1000, 2048)])
@pytest.mark.parametrize("bias", [False, True])
def test_gradients_of_confident_rows(N, K, d, dtype, bias):
    from clustering_flashassign_b200.soft import token_log_probs
    from test_logprob import reference, score_tol
    g = torch.Generator(device="cuda").manual_seed(N + d)
    T = TYPES[dtype]
    # a part common to all columns (scores near 30), and each column's own (13 for its rows)
    common = torch.randn(d, generator=g, device="cuda") * math.sqrt(30 / d)
    own = torch.randn(K, d, generator=g, device="cuda") * math.sqrt(13 / d)
    ids = torch.randint(0, K, (1, N), generator=g, device="cuda", dtype=torch.int32)
    c = (common + own).unsqueeze(0).to(T)
    x = (common + own[ids[0].long()]).unsqueeze(0).to(T)
    b = torch.zeros(1, K, device="cuda") if bias else None
    up = -(0.5 + torch.rand(1, N, generator=g, device="cuda"))
    leaves = [t.requires_grad_(True) for t in (x, c, b) if t is not None]
    r = token_log_probs(x, c, ids, bias=b)
    got = torch.autograd.grad([r.logp], leaves, [up])
    with torch.no_grad():
        s, lp, p, lse, logp, ent, A = reference(x, c, ids, 1.0, b)
        tol = score_tol(x, A, s).unsqueeze(-1)
        a = up.double().unsqueeze(-1)
        hot = torch.zeros_like(p).scatter_(-1, ids.long().unsqueeze(-1), 1.0)
        pt = (p * hot).sum(-1, keepdim=True)
        assert float((pt > 0.99).double().mean()) > 0.9  # the rows are confident
        # 1 - p without the cancellation
        rest = torch.where(hot > 0, -math.inf, lp).logsumexp(-1, keepdim=True).exp()
        G = torch.where(hot > 0, a * rest, -a * p)
        eG = a.abs() * torch.where(hot > 0, 4 * tol * rest + 2.0 ** -20, 4 * tol * p)
        step = torch.finfo(T).eps / 2
        two = N * K * d <= 2 ** 31 or N <= 64
        ground = step * step if two else step
        for i, (v, w_at) in enumerate(zip(got, (c, x, None))):
            if i == 2:
                want, bound = G.sum(1), eG.sum(1) + (N / 32 + 8) * U * G.abs().sum(1)
            else:
                M, E = (G, eG) if i == 0 else (G.transpose(1, 2), eG.transpose(1, 2))
                other = w_at.double()
                want, n = M @ other, M.shape[-1]
                lin = (ground + ((n / 16 + 20) + 4) * U)
                bound = (M.abs() @ other.abs()) * lin + E @ other.abs() + want.abs() * step
                if dtype == "fp16":  # subnormal results, and subnormal entries of the scaled G
                    bound = bound + 2.0 ** -25 + 6.0 * 2.0 ** -38 * other.abs().sum(1, keepdim=True)
            assert ((v.double() - want).abs() <= bound).all(), ("dx", "dc", "dbias")[i]
