"""Calls one after another on a stream, each reading what the one before wrote.

Kernels of the library start while their predecessor drains; a chain without a
synchronisation has to give what the same calls give one at a time.
"""
import pytest
import torch

import clustering_flashassign_b200 as fk
from clustering_flashassign_b200.soft import expert_mixture, token_log_probs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K,d", [(900, 300, 64), (5000, 700, 136), (40000, 1000, 128)])
def test_assign_log_probabilities_and_gradients(N, K, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(N)
    xs = [torch.randn(1, N, d, generator=g, device="cuda").to(dtype) for _ in range(4)]
    cs = [torch.randn(1, K, d, generator=g, device="cuda").to(dtype) for _ in range(4)]
    biases = [torch.randn(1, K, generator=g, device="cuda") for _ in range(4)]
    up = torch.randn(1, N, generator=g, device="cuda")
    x, c, bias = xs[0].clone(), cs[0].clone(), biases[0].clone()
    ids = torch.empty(1, N, device="cuda", dtype=torch.int32)
    o = torch.empty(4, 1, N, device="cuda")
    ti, tl = torch.empty(1, N, 3, device="cuda", dtype=torch.int32), torch.empty(1, N, 3, device="cuda")
    dx, dc, db = torch.empty_like(x), torch.empty_like(c), torch.empty_like(bias)

    def step(i, wait):
        sync = torch.cuda.synchronize if wait else (lambda: None)
        x.copy_(xs[i]), c.copy_(cs[i]), bias.copy_(biases[i])
        sync()
        fk.fk_assign(x, c, ids)
        sync()
        fk.fk_logprob(x, c, ids, o[0], o[1], o[2], ti, tl, bias=bias, scale=0.5, lse_rest=o[3])
        sync()
        fk.fk_logprob_backward(x, c, ids, o[1], o[2], up, None, up, dx, dc, db, bias=bias, scale=0.5, lse_rest=o[3])
        sync()
        fk.fk_logprob(dx, c, ti[..., 0].contiguous(), o[0], o[1], scale=0.5)
        sync()
        return [t.clone() for t in (ids, o, ti, tl, dx, dc, db)]

    want = [step(i, True) for i in range(4)]
    for _ in range(3):
        got = [step(i, False) for i in range(4)]
        for w, v in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, v))
    assert fk.fk_device_error() == fk.FK_OK


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,d,F", [(1, 16, 2, 512, 256), (5, 64, 4, 264, 136), (200, 8, 2, 128, 512),
                                       (64, 128, 8, 256, 96)])
def test_layers_of_experts(T, E, k, d, F, dtype):
    """Units of one warp and of several; every layer reads the one before.  (A layer squares
    the size of its rows, times 3 / sqrt(2): three layers reach 100, five leave fp16's range.)"""
    g = torch.Generator(device="cuda").manual_seed(T)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")

    layers = [((normal(E, d) / d ** 0.5).to(dtype), (normal(E, 2 * F, d) / d ** 0.5).to(dtype),
               (normal(E, d, F) * 3 / F ** 0.5).to(dtype)) for _ in range(3)]
    x = normal(T, d).to(dtype)

    def run(wait):
        out, h = [], x
        for w in layers:
            r = expert_mixture(h, *w, k)
            if wait:
                torch.cuda.synchronize()
            h = r.y
            out += list(r)
            out += list(token_log_probs(h, w[0], r.expert_ids[:, 0], top=2))
            if wait:
                torch.cuda.synchronize()
        return out

    want = run(True)
    assert torch.isfinite(want[-1]).all()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(want, run(False)))
    assert fk.fk_device_error() == fk.FK_OK
