"""The mixture-of-experts layer against the definition in fp64.

Tolerance per output value: half a step of the result's type; h held as hi + lo (2^-16
of each value for bf16, 2^-21 and 2^-19 absolute for fp16's h / 64); fp32 accumulation
of the two contractions, 32 elements to a step over 8 warps: at most
(len / 16 + 24) roundings of 2^-23 of the sum of absolute products, carried through
the activation (its slope is at most 1.13).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -23


def make(T, E, d, F, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, s=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * s).to(dtype)

    return (normal(T, d), normal(E, d, s=1.5 / math.sqrt(d)), normal(E, 2 * F, d, s=1 / math.sqrt(d)),
            normal(E, d, F, s=1 / math.sqrt(F)))


def reference(x, router, w_in, w_out, k, renorm, act):
    T, d = x.shape
    F = w_out.shape[2]
    xd = x.double()
    s = xd @ router.double().T
    order = torch.sort(s, dim=1, descending=True, stable=True)
    ids = order.indices[:, :k]
    p = torch.softmax(s, 1).gather(1, ids)
    w = p / p.sum(1, keepdim=True) if renorm else p
    f = torch.nn.functional.silu if act == "silu" else torch.nn.functional.gelu
    y, tol = torch.zeros_like(xd), torch.zeros_like(xd)
    bf = x.dtype == torch.bfloat16
    for j in range(k):
        for t in range(T):
            e = ids[t, j]
            wi, wo = w_in[e].double(), w_out[e].double()
            u, au = wi @ xd[t], wi.abs() @ xd[t].abs()
            g, up = u[:F], u[F:]
            h = f(g) * up
            du = (d / 16 + 24) * U * au
            dh = 1.13 * du[:F] * up.abs() + g.abs() * du[F:] + 8 * U * h.abs()
            dh = dh + h.abs() * (2.0 ** -16 if bf else 2.0 ** -21) + (0 if bf else 2.0 ** -19)
            y[t] += w[t, j] * (wo @ h)
            tol[t] += w[t, j] * (wo.abs() @ (dh + (F / 16 + 24) * U * 2 * h.abs()))
    T_eps = torch.finfo(x.dtype).eps / 2
    return y, tol + y.abs() * (T_eps + 8 * U) + (0 if bf else 2.0 ** -25), ids, w


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [
    # T, E, k, d, F
    (1, 1, 1, 8, 8), (1, 4, 2, 64, 16), (3, 5, 5, 72, 40), (8, 8, 2, 256, 136), (9, 33, 16, 128, 24),
    (40, 3, 1, 264, 264), (17, 512, 8, 40, 16), (130, 6, 3, 96, 56), (256, 2, 2, 24, 32), (1, 64, 8, 1024, 512),
], ids=str)
def test_layer_matches_the_definition(shape, dtype):
    import clustering_flashassign_b200 as fk
    from clustering_flashassign_b200.soft import expert_mixture
    T, E, k, d, F = shape
    x, router, w_in, w_out = make(T, E, d, F, TYPES[dtype], seed=T + E + d)
    for renorm, act in ((True, "silu"), (False, "gelu")):
        r = expert_mixture(x, router, w_in, w_out, k, renormalize=renorm, activation=act)
        y, tol, ids, w = reference(x, router, w_in, w_out, k, renorm, act)
        assert torch.equal(r.expert_ids.long(), ids)
        # scores are exact to fp64; exp, the sum over E and the division: fp32
        assert ((r.expert_weights - w).abs() <= w * (E / 32 + 16) * U).all()
        assert ((r.y.double() - y).abs() <= tol).all()
    assert fk.fk_device_error() == fk.FK_OK


def test_many_tokens_of_one_expert_and_repeats_are_reproducible():
    from clustering_flashassign_b200.soft import expert_mixture
    x, router, w_in, w_out = make(100, 16, 512, 256, torch.bfloat16, seed=3)
    x[:, 0] = 20.0
    router[5, 0] = 3.0  # every token's first choice
    first = expert_mixture(x, router, w_in, w_out, 4)
    assert (first.expert_ids[:, 0] == 5).all()
    for _ in range(5):
        again = expert_mixture(x, router, w_in, w_out, 4)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    y, tol, _, _ = reference(x, router, w_in, w_out, 4, True, "silu")
    assert ((first.y.double() - y).abs() <= tol).all()


def test_ties_nan_rows_and_empty_batches():
    from clustering_flashassign_b200.soft import expert_mixture
    x, router, w_in, w_out = make(6, 40, 64, 32, torch.bfloat16, seed=4)
    router[:] = router[0].clone()  # every score is equal
    clean = expert_mixture(x, router, w_in, w_out, 3)
    assert (clean.expert_ids == torch.tensor([0, 1, 2], device="cuda", dtype=torch.int32)).all()
    x[2] = float("nan")
    r = expert_mixture(x, router, w_in, w_out, 3)
    assert torch.isnan(r.y[2]).all() and torch.isnan(r.expert_weights[2]).all()
    assert ((r.expert_ids >= 0) & (r.expert_ids < 40)).all()
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(r.y[keep], clean.y[keep])
    empty = expert_mixture(x[:0], router, w_in, w_out, 3)
    assert empty.y.shape == (0, 64) and empty.expert_ids.shape == (0, 3)
