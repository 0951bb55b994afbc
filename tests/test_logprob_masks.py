"""Finite masks, and scores so large that fp32 holds whole numbers only.

A bias beyond 2.3e38 in magnitude counts as that (a score in base 2 must not overflow);
beside an ordinary column either contributes exactly nothing.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -23
LOWEST = [-1e9, -1e30, torch.finfo(torch.bfloat16).min, torch.finfo(torch.float32).min]


def run(x, c, ids, bias, top, up):
    from clustering_flashassign_b200.soft import token_log_probs
    leaves = [t.clone().requires_grad_(True) for t in (x, c, bias)]
    r = token_log_probs(leaves[0], leaves[1], ids, bias=leaves[2], top=top)
    return r, torch.autograd.grad([r.logp, r.lse, r.entropy], leaves, up)


@pytest.mark.parametrize("value", LOWEST, ids=lambda v: f"{v:.0e}")
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N", [9, 300])
def test_a_finite_mask_does_what_an_infinite_one_does(N, dtype, value):
    """All results of open columns are those of a bias of -inf, bit for bit."""
    from test_logprob import make
    x, c, ids, _ = make(2, N, 500, 72, TYPES[dtype], seed=N)
    g = torch.Generator(device="cuda").manual_seed(1)
    masked = torch.rand(2, 500, generator=g, device="cuda") < 0.4
    masked[:, 3] = False
    ids = torch.where(masked.gather(1, ids.clamp(min=0).long()), 3, ids).int()
    bias = torch.randn(2, 500, generator=g, device="cuda")
    up = [torch.randn(2, N, generator=g, device="cuda") * v for v in (1.0, 0.1, 9.0)]
    want, dwant = run(x, c, ids, bias.masked_fill(masked, -math.inf), 5, up)
    got, dgot = run(x, c, ids, bias.masked_fill(masked, value), 5, up)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    for a, b in zip(dwant, dgot):
        assert torch.isfinite(b).all() and torch.equal(a, b)


@pytest.mark.parametrize("value", LOWEST, ids=lambda v: f"{v:.0e}")
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N", [9, 300])
def test_rows_whose_every_column_has_the_lowest_bias_are_even(N, dtype, value):
    """The products vanish beside the bias (fp32 steps of 64 and more): p = 1 / K."""
    from test_logprob import make
    K = 500
    x, c, ids, _ = make(2, N, K, 72, TYPES[dtype], seed=N, gain=1.0)
    bias = torch.zeros(2, K, device="cuda")
    bias[1] = value
    up = [torch.ones(2, N, device="cuda") for _ in range(3)]
    up[1].zero_()
    r, (dx, dc, db) = run(x, c, ids, bias, 3, up)
    valid = ids[1] >= 0
    assert torch.isfinite(r.lse).all()
    # log2 of the sum (1 ulp of 8 to 16), its conversion, and the exponentials
    assert ((r.logp[1] + math.log(K))[valid].abs() <= 16 * U * math.log(K)).all()
    assert ((r.entropy[1] - math.log(K)).abs() <= 16 * U * math.log(K)).all()
    count = max(value, -2.3e38)
    assert ((r.lse[1] - count).abs() <= 2 * U * abs(count)).all()
    assert ((r.top_logp[1] + math.log(K)).abs() <= 16 * U * math.log(K)).all()
    # p from lse: held to 2^-47 of its size (up to 2^31 in base 2), beyond that from the entropy
    rel = 2.0 ** -15
    G = -torch.ones(N, K, device="cuda", dtype=torch.float64) / K
    G.scatter_add_(1, ids[1].clamp(min=0).long().unsqueeze(1), torch.ones(N, 1, device="cuda", dtype=torch.float64))
    # entropy's term vanishes where p is even: p (log p + H) = 0
    G[~valid] = 0
    eG = torch.full_like(G, 1 / K) * rel * (2 + math.log(K))
    step = torch.finfo(TYPES[dtype]).eps / 2 if dtype != "fp32" else U
    for v, want, bound in ((dx[1], G @ c[1].double(), eG @ c[1].double().abs() + (G.abs() @ c[1].double().abs()) * (step + 200 * U)),
                           (dc[1], G.T @ x[1].double(), eG.T @ x[1].double().abs() + (G.abs().T @ x[1].double().abs()) * (step + 200 * U)),
                           (db[1], G.sum(0), eG.sum(0) + G.abs().sum(0) * (N / 32 + 8) * U)):
        assert ((v.double() - want).abs() <= bound + want.abs() * step + 2.0 ** -25).all()
    assert torch.isfinite(dx[0]).all() and torch.isfinite(dc[0]).all()


def test_nan_and_infinite_biases_are_not_hidden():
    from clustering_flashassign_b200.soft import token_log_probs
    from test_logprob import make
    x, c, ids, _ = make(1, 20, 100, 32, torch.float16)
    for bad in (math.nan, math.inf):
        bias = torch.zeros(1, 100, device="cuda")
        bias[0, 7] = bad
        r = token_log_probs(x, c, ids.clamp(min=0), bias=bias)
        assert not torch.isfinite(r.lse).any() and torch.isnan(r.entropy).all()


@pytest.mark.parametrize("shift", [-1e30, 1e30, 3e38])
@pytest.mark.parametrize("N,top", [(5, 3), (5, 0), (200, 0), (5000, 3), (5000, 15)])
def test_equal_biases_beyond_the_range_of_scores(shift, N, top):
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
    # p from lse, held to 2^-47 of its size (up to 2^31 in base 2), and fp32 sums of N terms
    assert ((db[0].double() - want).abs() <= N / K * 2.0 ** -15 + (count + N / K) * (N / 32 + 8) * U).all()
    assert (dc == 0).all()


@pytest.mark.parametrize("temperature", [1.0, 1e-3, 1e-6, 1e-9, 1e-12, 1e-20])
@pytest.mark.parametrize("N", [40, 5000])
def test_low_temperatures_pick_the_nearest_centroid(N, temperature):
    """Large products and a large bias that nearly cancel: neither may be cut on its own."""
    from clustering_flashassign_b200.soft import token_log_probs
    K, d = 200, 48
    g = torch.Generator(device="cuda").manual_seed(N)
    c = torch.randn(1, K, d, generator=g, device="cuda")
    c *= 1 + 3 * torch.rand(1, K, 1, generator=g, device="cuda")  # of lengths 7 to 28: x.c alone misleads
    near = torch.randint(0, K, (N,), generator=g, device="cuda")
    x = (c[:, near] + 0.05 * torch.randn(1, N, d, generator=g, device="cuda")).contiguous()
    bias = -c.square().sum(-1) / temperature
    leaf = x.clone().requires_grad_(True)
    r = token_log_probs(leaf, c, near.int().unsqueeze(0), scale=2 / temperature, bias=bias, top=2)
    d2 = torch.cdist(x.double(), c.double()).square()
    assert (d2.argmin(-1)[0] == near).all()
    assert torch.equal(r.top_ids[0, :, 0].long(), near)
    # every other centroid is at least 20 further off (squared): p < 200 e^-20
    gap = d2.topk(2, dim=-1, largest=False).values
    assert float((gap[..., 1] - gap[..., 0]).min()) > 20
    assert (r.logp.abs() <= 200 * math.exp(-20)).all() and (r.entropy.abs() <= 40 * 200 * math.exp(-20) + 16 * U).all()
    dx = torch.autograd.grad(r.logp.sum(), leaf)[0]
    # scale (1 - p) |c| with 1 - p off by two exponentials (2^-20)
    assert (dx.abs() <= 2 / temperature * (200 * math.exp(-20) + 2.0 ** -20) * 2 * float(c.abs().max())).all()
