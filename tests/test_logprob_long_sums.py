"""Gradients whose contraction is long and whose terms have one sign: a truncating chain of
tensor-core accumulations shows as a bias, which half a step of the result's type hides
in single values and the mean over all values does not.

Bound of the mean relative error: segments of 4096 terms lose at most (4096 / 16 + 16)
units of 2^-23, adding them up half a unit each; roundings to nearest of G and of the
result average out over millions of values (2^-17 is left for them).
"""
import math

import pytest
import torch

import clustering_flashassign_b200 as fk

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("N,K,d", [(4096, 131072, 1024),   # dx: 131072 terms in two parts
                                   (40000, 20000, 1024)])  # dc: 40000 terms
def test_long_sums_of_one_sign(N, K, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.rand(1, N, d, generator=g, device="cuda") * 0.02 + 0.01).to(dtype)
    c = (torch.rand(1, K, d, generator=g, device="cuda") * 0.5 + 0.5).to(dtype)
    ids = torch.full((1, N), -1, device="cuda", dtype=torch.int32)
    o = torch.empty(3, 1, N, device="cuda")
    fk.fk_logprob(x, c, ids, o[0], o[1], lse_rest=o[2])
    up = torch.full((1, N), 64.0, device="cuda")
    dx, dc = torch.empty_like(x), torch.empty_like(c)
    fk.fk_logprob_backward(x, c, ids, o[1], dlse=up, dx=dx, dc=dc, lse_rest=o[2])
    want_dc = torch.zeros(K, d, device="cuda", dtype=torch.float64)
    off = []
    for n in range(0, N, 2048):
        p = torch.softmax(x[0, n:n + 2048].double() @ c[0].double().T, 1) * 64
        w = p @ c[0].double()
        off.append(((dx[0, n:n + 2048].double() - w) / w).mean())
        want_dc += p.T @ x[0, n:n + 2048].double()
    off_dc = ((dc[0].double() - want_dc) / want_dc).mean()

    def bound(terms):
        return (4096 / 16 + 16 + math.ceil(terms / 4096) / 2) * U + 2.0 ** -17

    assert abs(float(off_dc)) <= bound(N)
    if dtype == torch.float16:  # bf16: the roundings of a row's nearly equal p do not average out
        assert abs(float(torch.stack(off).mean())) <= bound(K)
