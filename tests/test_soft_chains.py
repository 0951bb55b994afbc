"""Calls one after another on a stream, each reading what the one before wrote.

Kernels of the library start while their predecessor drains; a chain without a
synchronisation has to give what the same calls give one at a time.
"""
import pytest
import torch

import clustering_flashassign_b200 as fk

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
