"""The mixture-of-experts layer where the hidden activations are small, or overflow.

Tolerance per output value, against the definition in fp64: half a step of the result's
type; fp32 accumulation as in test_moe.py; h held in two parts of the weights' type.
For fp16 the second part is kept at 2^11 times its size: the pair resolves 2^-21 of h,
or, where h / 64 and that part are subnormal, steps of 2^-24 / 2^11 * 64, so half of
2^-29 absolute.  Nothing else of h is lost, however small the inputs are.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -23


def definition(x, router, w_in, w_out, k, act):
    xd, F = x.double(), w_out.shape[2]
    p = torch.softmax(xd @ router.double().T, 1)
    best = torch.sort(p, dim=1, descending=True, stable=True)
    ids = best.indices[:, :k]
    w = best.values[:, :k] / best.values[:, :k].sum(1, keepdim=True)
    f = torch.nn.functional.silu if act == "silu" else torch.nn.functional.gelu
    bf, d = x.dtype == torch.bfloat16, x.shape[1]
    y, tol = torch.zeros_like(xd), torch.zeros_like(xd)
    for t in range(x.shape[0]):
        for j in range(k):
            wi, wo = w_in[ids[t, j]].double(), w_out[ids[t, j]].double()
            u, au = wi @ xd[t], wi.abs() @ xd[t].abs()
            h = f(u[:F]) * u[F:]
            du = (d / 16 + 24) * U * au
            dh = 1.13 * du[:F] * u[F:].abs() + f(u[:F]).abs() * du[F:] + 8 * U * h.abs()
            dh = dh + (h.abs() * 2.0 ** -16 if bf else h.abs() * 2.0 ** -21 + 2.0 ** -30)
            y[t] += w[t, j] * (wo @ h)
            tol[t] += w[t, j] * (wo.abs() @ (dh + (F / 16 + 24) * U * 2 * h.abs()))
    step = torch.finfo(x.dtype).eps / 2
    return y, tol + y.abs() * (step + 8 * U) + (0 if bf else 2.0 ** -25)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("scale", [0.1, 0.03, 1e-2, 3e-3, 1e-3])
@pytest.mark.parametrize("shape", [(2, 4, 2, 512, 256), (40, 3, 2, 264, 136)], ids=str)
def test_small_hidden_activations_keep_their_digits(shape, scale, act, dtype):
    from clustering_flashassign_b200.soft import expert_mixture
    T, E, k, d, F = shape
    g = torch.Generator(device="cuda").manual_seed(T + d)

    def normal(*size, s=1.0):
        return (torch.randn(*size, generator=g, device="cuda") * s).to(TYPES[dtype])

    x, router = normal(T, d, s=scale), normal(E, d)
    w_in, w_out = normal(E, 2 * F, d, s=1 / math.sqrt(d)), normal(E, d, F)
    r = expert_mixture(x, router, w_in, w_out, k, activation=act)
    y, tol = definition(x, router, w_in, w_out, k, act)
    assert ((r.y.double() - y).abs() <= tol).all()


@pytest.mark.parametrize("dtype,big", [("fp16", 4096.0), ("bf16", 1e18)])
def test_hidden_activations_beyond_the_range_give_infinities(dtype, big):
    """h of 2^24 and more in fp16 (results beyond 65504), 1e40 in bf16 (beyond fp32): the result is infinite."""
    from clustering_flashassign_b200.soft import expert_mixture
    T, d, F = 3, 64, 32
    x = torch.zeros(T, d, device="cuda")
    x[:, 0] = 1.0
    x[1, 0] = big
    w_in = torch.zeros(1, 2 * F, d, device="cuda")
    w_in[:, :, 0] = 1.0 if dtype == "fp16" else 100.0
    w_out = torch.ones(1, d, F, device="cuda")
    w_out[:, 1::2] = -1.0
    x, w_in, w_out = (t.to(TYPES[dtype]) for t in (x, w_in, w_out))
    router = torch.zeros(1, d, device="cuda", dtype=TYPES[dtype])
    y = expert_mixture(x, router, w_in, w_out, 1).y
    assert (y[1, 0::2] == math.inf).all() and (y[1, 1::2] == -math.inf).all()
    assert torch.isfinite(y[[0, 2]]).all()
