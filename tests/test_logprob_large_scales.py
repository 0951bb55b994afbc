"""Scales so large (temperatures so low) that scores leave what fp32 holds to a unit,
without a bias: the products are rounded the same way wherever they are used."""
import math

import pytest
import torch

import clustering_flashassign_b200 as fk

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -23


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("scale", [1e3, 1e6, 3e7, 1e9, 1e12, 1e20, 1e30])
@pytest.mark.parametrize("N,K,top", [(40, 200, 3), (300, 3000, 0), (5000, 200, 3), (5000, 200, 20)])
def test_the_largest_score_takes_all(N, K, top, scale, dtype):
    from clustering_flashassign_b200.soft import token_log_probs
    d = 80
    g = torch.Generator(device="cuda").manual_seed(N)
    c = torch.randn(1, K, d, generator=g, device="cuda")
    c = (c / c.norm(dim=-1, keepdim=True)).to(TYPES[dtype])
    near = torch.randint(0, K, (1, N), generator=g, device="cuda")
    x = (c[0, near[0]].float() + 0.03 * torch.randn(N, d, generator=g, device="cuda")).unsqueeze(0).to(TYPES[dtype])
    s = x.double() @ c.double().transpose(1, 2)
    best = s.topk(2, dim=-1)
    assert torch.equal(best.indices[..., 0], near)
    gap = float((best.values[..., 0] - best.values[..., 1]).min())
    assert gap * 1e3 > 100  # p of every other column is below e^-100
    leaves = [x.clone().requires_grad_(True), c.clone().requires_grad_(True)]
    r = token_log_probs(leaves[0], leaves[1], near.int(), scale=scale, top=top)
    # the entropy: log2 of a sum below 2 and the mean below 4 of base-2 differences, each rounded
    assert (r.logp.abs() <= 1e-30).all() and (r.entropy.abs() <= 16 * U).all()
    assert ((r.lse - scale * best.values[..., 0]).abs() <= 64 * U * scale * best.values[..., 0]).all()
    if top:
        assert torch.equal(r.top_ids[..., 0].long(), near)
        assert (r.top_logp[..., 0].abs() <= 1e-30).all() and (r.top_logp[..., 1:] < -100).all()
    # 1 - p is off by the exponentials (2^-20); gradients that leave the type's range are not looked at
    if scale <= 1e9 or dtype != "fp16":
        dx, dc = torch.autograd.grad([r.logp.sum() + r.entropy.sum()], leaves)
        count = torch.bincount(near[0], minlength=K).view(1, K, 1)
        assert (dx.double().abs() <= scale * 2.0 ** -18 * float(c.abs().max())).all()
        assert (dc.double().abs() <= scale * 2.0 ** -18 * count * float(x.abs().max())).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("scale", [1e6, 1e9, 1e20, 1e30])
@pytest.mark.parametrize("N", [30, 5000])
def test_equal_products_share(N, scale, dtype):
    """Four copies of every column: the largest score is met four times, and p = 1 / 4."""
    from clustering_flashassign_b200.soft import token_log_probs
    d, K = 48, 60
    g = torch.Generator(device="cuda").manual_seed(N)
    base = torch.randn(1, K, d, generator=g, device="cuda")
    base = base / base.norm(dim=-1, keepdim=True)
    c = base.repeat(1, 4, 1).to(TYPES[dtype]).contiguous()
    near = torch.randint(0, K, (1, N), generator=g, device="cuda")
    x = (base[0, near[0]] * 0.9).unsqueeze(0).to(TYPES[dtype])
    leaf = c.clone().requires_grad_(True)
    r = token_log_probs(x, leaf, (near + K).int(), scale=scale, top=4)
    assert ((r.logp + math.log(4)).abs() <= 16 * U).all() and ((r.entropy - math.log(4)).abs() <= 16 * U).all()
    assert torch.equal(r.top_ids.long(), torch.stack([near + i * K for i in range(4)], -1))
    assert ((r.top_logp + math.log(4)).abs() <= 16 * U).all()
    if dtype == "fp32" or scale <= 1e6:
        up = 1e-3 / scale
        dc = torch.autograd.grad(r.logp, leaf, [torch.full_like(r.logp, up)])[0].double()
        xs = x.double()[0]
        want = torch.zeros(4 * K, d, device="cuda", dtype=torch.float64)
        for i in range(4):
            want.index_add_(0, near[0] + i * K, xs * ((1.0 if i == 1 else 0.0) - 0.25))
        want *= scale * up
        size = torch.zeros(4 * K, 1, device="cuda", dtype=torch.float64).index_add_(
            0, (near[0].unsqueeze(0) + K * torch.arange(4, device="cuda").unsqueeze(1)).reshape(-1),
            xs.abs().amax(-1, keepdim=True).repeat(4, 1))
        # G rounded to the type (relative 2^-9 at worst), p from lse held to 2^-47 of its size (up to 2^31)
        assert ((dc[0] - want).abs() <= 1e-3 * size * (2.0 ** -8 + 2.0 ** -14) + 2.0 ** -25).all()


def test_scales_that_overflow_in_base_2_are_refused():
    from clustering_flashassign_b200.soft import token_log_probs
    x = torch.randn(1, 4, 16, device="cuda")
    ids = torch.zeros(1, 4, device="cuda", dtype=torch.int32)
    with pytest.raises(fk.FkError, match="scale"):
        token_log_probs(x, x, ids, scale=3e38)
