"""Log probabilities and gradients at the sizes that CTA pairs work on: two rounds of
128 x 256 tiles for all SMs (296), or few tiles of 128 K-blocks and more; and the joins
of many rows with many partial results.  Definition and tolerances: test_logprob.py."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -23


def check_forward(B, N, K, d, dtype, tops, biases, seed=0):
    from clustering_flashassign_b200.soft import token_log_probs
    from test_logprob import make, reference, score_tol
    for bias in biases:
        x, c, ids, b = make(B, N, K, d, TYPES[dtype], seed=seed, bias=bias)
        s, lp, p, lse, logp, ent, A = reference(x, c, ids, 0.7, b)
        del p
        tol = score_tol(x, A, s)
        fin = torch.isfinite(logp)
        order = torch.topk(s, max(max(tops), 1) + 1, dim=-1)  # no ties: random scores in fp64
        for top in tops:
            r = token_log_probs(x, c, ids, scale=0.7, bias=b, top=top)
            assert ((r.lse - lse).abs() <= 2 * tol).all()
            assert torch.equal(torch.isfinite(r.logp), fin)
            assert ((r.logp - logp).abs()[fin] <= 3 * tol[fin]).all()
            assert ((r.entropy - ent).abs() <= 4 * tol * (1 + math.log(K)) + 8 * U * (ent + 1)).all()
            if top:
                assert torch.equal(r.top_ids.long(), order.indices[..., :top])
                want = order.values[..., :top] - lse.unsqueeze(-1)
                assert ((r.top_logp - want).abs() <= 3 * tol.unsqueeze(-1)).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N,K,d", [
    (2100, 9000, 1032),  # pairs, segments, a block per row
    (4200, 9000, 200),   # pairs, one chain (fp32: segments), 12 partial results a row
    (300, 600, 1500),    # fp32: pairs of a deep contraction (16-bit: single CTAs, d 1504)
    (92, 326, 3250),     # the same with fewer rows than one CTA holds
], ids=str)
@pytest.mark.parametrize("bias", [None, "plain", "mask"])
def test_statistics_and_alternatives_of_pairs(N, K, d, dtype, bias):
    if dtype != "fp32":
        d = (d + 7) // 8 * 8
    check_forward(1, N, K, d, dtype, (0, 4, 12, 20), (bias,), seed=N + d)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_deep_rows_of_16_bits_and_batches(dtype):
    check_forward(1, 130, 300, 8200, dtype, (0, 5), (None, "plain"))    # 129 K-blocks and more: pairs
    check_forward(5, 600, 3000, 136, dtype, (0, 3, 8), (None, "mask"))  # pairs, batch by batch


@pytest.mark.parametrize("B,N,K,d", [(1, 5000, 40000, 64),     # 33 partial results a row
                                     (15, 300, 20000, 40)],    # 81
                         ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_joins_of_many_rows_with_many_partial_results(B, N, K, d, dtype):
    check_forward(B, N, K, d, dtype, (1, 5, 10, 14, 28), (None, "plain") if B == 1 else ("mask",))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N,K,d", [(1100, 9000, 264),   # above 2^31 products: G in one part, by pairs
                                   (1100, 9000, 1032),  # and segments
                                   (92, 326, 3250)], ids=str)
@pytest.mark.parametrize("bias", [None, "plain", "mask"])
def test_gradients_of_pairs(N, K, d, dtype, bias):
    from clustering_flashassign_b200.soft import token_log_probs
    from test_logprob import make, reference_grads
    if dtype != "fp32":
        d = (d + 7) // 8 * 8
    T = TYPES[dtype]
    x, c, ids, b = make(1, N, K, d, T, seed=N + K + d, bias=bias)
    g = torch.Generator(device="cuda").manual_seed(5)
    up = [torch.randn(1, N, generator=g, device="cuda") * v for v in (1.0, 0.1, 0.3)]
    if bias == "mask":
        up[0][b.gather(1, ids.clamp(min=0).long()) == -math.inf] = 0.0
    leaves = [t.requires_grad_(True) for t in (x, c, b) if t is not None]
    r = token_log_probs(x, c, ids, scale=0.7, bias=b)
    got = torch.autograd.grad([r.logp, r.lse, r.entropy], leaves, up)
    with torch.no_grad():
        want, absG, tol = reference_grads(x, c, ids, 0.7, b, up)
        step = torch.finfo(T).eps / 2
        ground = 2.0 ** -25 if dtype == "fp32" else step
        pairs = 6 if dtype == "fp32" else 1
        eG = absG * (4 * tol * (1 + math.log(K))).unsqueeze(-1)
        for i, (a, w) in enumerate(zip(got, want)):
            if i == 2:
                bound = eG.sum(1) + absG.sum(1) * (N / 32 + 8) * U
                assert ((a - w).abs() <= bound + 1e-30).all(), "dbias"
                continue
            other = (c if i == 0 else x).detach().double().abs()
            M = absG if i == 0 else absG.transpose(1, 2)
            E = eG if i == 0 else eG.transpose(1, 2)
            n = M.shape[-1]
            bound = 0.7 * (M @ other) * (ground + ((n / 16 + 20) * pairs + 4) * U) + 0.7 * (E @ other) + w.abs() * step
            if dtype == "fp16":
                big = absG.sum(-1).amax() * 4 + 1
                bound = bound + 2.0 ** -25 + 0.7 * big * 2.0 ** -38 * other.sum(1, keepdim=True)
            assert ((a.double() - w).abs() <= bound).all(), ("dx", "dc")[i]
