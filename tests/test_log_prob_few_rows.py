"""FlashKMeans.log_prob of fewer rows than centroids, and of none."""
import pytest
import torch

from clustering_flashassign_b200.kmeans import FlashKMeans

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [0, 1, 5, 11])
@pytest.mark.parametrize("batched", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_log_prob_of_fewer_rows_than_centroids(rows, batched, dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    data = torch.randn((3, 500, 32) if batched else (500, 32), generator=g, device="cuda").to(dtype)
    km = FlashKMeans(d=32, k=12, niter=5, dtype=dtype)
    km.train(data)
    few = data[..., :rows, :]
    r = km.log_prob(few, temperature=2.0, top=2)
    whole = km.log_prob(data, temperature=2.0, top=2)
    assert r.logp.shape == few.shape[:-1]
    # the nearest centroid is the likeliest one; the same rows score the same in a longer call
    # (fp32 sums whose joining order may differ: a few roundings of scores up to a few hundred)
    assert torch.equal(r.logp, r.top_logp[..., 0])
    c = km.centroids.to(dtype).double()
    d2 = torch.cdist(few.double(), c) ** 2
    want = torch.log_softmax(-d2 / 2.0, -1)
    if rows:
        tol = 2.0 ** -23 * 64 * float(d2.max())
        assert (r.logp - want.amax(-1)).abs().max() <= tol
        assert (r.logp - whole.logp[..., :rows]).abs().max() <= 2 * tol
    asked = km.log_prob(few, ids=torch.zeros(few.shape[:-1], device="cuda", dtype=torch.int64), temperature=2.0)
    assert asked.logp.shape == few.shape[:-1]


def test_log_prob_of_few_rows_is_differentiable():
    data = torch.randn(400, 32, device="cuda", dtype=torch.float16)
    km = FlashKMeans(d=32, k=12, niter=5)
    km.train(data)
    few = data[:3].clone().requires_grad_(True)
    grad = torch.autograd.grad(km.log_prob(few, temperature=2.0).logp.sum(), few)[0]
    more = data[:40].clone().requires_grad_(True)
    want = torch.autograd.grad(km.log_prob(more, temperature=2.0).logp[:3].sum(), more)[0][:3]
    # fp16 results of the same sums, G rounded by 2^-22 (two parts)
    assert (grad.double() - want.double()).abs().max() <= 2 * 2.0 ** -10 * want.abs().max()
