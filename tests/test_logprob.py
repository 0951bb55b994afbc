"""Token log probabilities and their gradients against the definition in fp64.

Tolerances, per row n and for operands whose products are exact in fp32 (fp16, bf16):
a score's fp32 accumulation over d terms in steps of 16 is off by at most
(d / 16 + 16) roundings of 2^-23 of A = scale * sum_j |x_j c_kj|; its base-2 form, the
exponential (2 ulp) and the sums add a few 2^-23 of |score| and of 1.  fp32 operands
as three bf16 parts add 2^-23 of A and six times the accumulation steps.  Gradients
carry, relative to sum |G| |operand|: half a step of the type G is rounded to, the
same accumulation bound over their contraction, and the score's error; the result is
rounded by half a step of its type.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -23


def make(B, N, K, d, dtype, seed=0, bias=None, ignore=0.2, gain=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randn(B, K, d, generator=g, device="cuda") * (gain / math.sqrt(d))
    x = torch.randn(B, N, d, generator=g, device="cuda")
    ids = torch.randint(0, K, (B, N), generator=g, device="cuda", dtype=torch.int32)
    ids[torch.rand(B, N, generator=g, device="cuda") < ignore] = -1
    b = None
    if bias:
        b = torch.randn(B, K, generator=g, device="cuda")
        if bias == "mask":
            b[torch.rand(B, K, generator=g, device="cuda") < 0.3] = -math.inf
    return x.to(dtype), c.to(dtype), ids, b


def reference(x, c, ids, scale, bias):
    xd, cd = x.double(), c.double()
    s = scale * (xd @ cd.transpose(1, 2))
    A = scale * (xd.abs() @ cd.abs().transpose(1, 2)).amax(-1)
    if bias is not None:
        b = bias.double().unsqueeze(1)
        s = torch.where(b == -math.inf, b, s + b)
    lse = torch.logsumexp(s, -1)
    lp = s - lse.unsqueeze(-1)
    p = lp.exp()
    ent = torch.special.entr(p).sum(-1)
    valid = ids >= 0
    logp = lp.gather(-1, ids.clamp(min=0).long().unsqueeze(-1)).squeeze(-1)
    return s, lp, p, lse, torch.where(valid, logp, 0.0), ent, A


def score_tol(x, A, s):
    d = x.shape[-1]
    steps = (d / 16 + 16) * (6 if x.dtype == torch.float32 else 1) + (2 if x.dtype == torch.float32 else 0)
    top = torch.where(torch.isfinite(s), s.abs(), 0.0).amax(-1)
    return steps * U * A + 8 * U * (top + 4)


SHAPES = [
    (1, 1, 1, 8), (1, 1, 2, 16), (1, 3, 7, 8), (2, 5, 255, 24), (1, 127, 256, 64), (1, 128, 257, 72),
    (1, 129, 1000, 128), (3, 200, 513, 40), (1, 300, 5003, 256), (1, 7, 33000, 512), (1, 1, 32000, 1024),
    (1, 2050, 700, 136),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_statistics_match_the_definition(shape, dtype):
    import clustering_flashassign_b200 as fk
    from clustering_flashassign_b200.soft import token_log_probs
    B, N, K, d = shape
    if dtype == "fp32":
        d += 3  # rows of any length
    for bias in (None, "plain", "mask"):
        if bias == "mask" and K < 16:
            continue
        x, c, ids, b = make(B, N, K, d, TYPES[dtype], seed=B + N + K + d, bias=bias)
        top = min(K, 5)
        r = token_log_probs(x, c, ids, scale=0.7, bias=b, top=top)
        s, lp, p, lse, logp, ent, A = reference(x, c, ids, 0.7, b)
        tol = score_tol(x, A, s)
        assert ((r.lse - lse).abs() <= 2 * tol).all()
        fin = torch.isfinite(logp)
        assert torch.equal(torch.isfinite(r.logp), fin)
        assert ((r.logp - logp).abs()[fin] <= 3 * tol[fin]).all()
        # entropy: the scores' errors weighted by p (1 + |log p|), and fp32 sums of K terms
        assert ((r.entropy - ent).abs() <= 4 * tol * (1 + math.log(K)) + 8 * U * (ent + 1)).all()
        want = torch.sort(s, dim=-1, descending=True, stable=True)
        assert torch.equal(r.top_ids.long(), want.indices[..., :top])
        assert ((r.top_logp - lp.gather(-1, want.indices[..., :top])).abs() <= 3 * tol.unsqueeze(-1)).all()
    assert fk.fk_device_error() == fk.FK_OK


def reference_grads(x, c, ids, scale, bias, up):
    s, lp, p, lse, logp, ent, A = reference(x, c, ids, scale, bias)
    z = torch.zeros_like(lse)
    a, l, e = (z if u is None else u.double() for u in up)
    a = torch.where(ids >= 0, a, 0.0).unsqueeze(-1)
    l, e = l.unsqueeze(-1), e.unsqueeze(-1)
    lpf = lp.clamp(min=-1e4)
    G = p * (l - a - e * (lpf + ent.unsqueeze(-1)))
    absG = p * (l.abs() + a.abs() + e.abs() * (lpf.abs() + ent.unsqueeze(-1)))
    hot = torch.zeros_like(p).scatter_(-1, ids.clamp(min=0).long().unsqueeze(-1), 1.0) * (ids >= 0).unsqueeze(-1)
    G = G + hot * a
    absG = absG + hot * a.abs()
    if bias is not None:
        keep = (bias != -math.inf).unsqueeze(1)
        G, absG = torch.where(keep, G, 0.0), torch.where(keep, absG, 0.0)
    xd, cd = x.double(), c.double()
    tol = score_tol(x, A, s)
    return (scale * G @ cd, scale * G.transpose(1, 2) @ xd, G.sum(1)), absG, tol


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(1, 1, 2, 8), (1, 5, 33, 16), (2, 130, 257, 72), (1, 129, 1000, 128),
                                   (3, 40, 513, 264), (1, 700, 3001, 256), (1, 2050, 130, 40)], ids=str)
@pytest.mark.parametrize("bias", [None, "plain", "mask"])
def test_gradients_match_the_formula(shape, dtype, bias):
    import clustering_flashassign_b200 as fk
    from clustering_flashassign_b200.soft import token_log_probs
    B, N, K, d = shape
    if bias == "mask" and K < 16:
        pytest.skip("too few columns to mask")
    if dtype == "fp32":
        d += 3
    x, c, ids, b = make(B, N, K, d, TYPES[dtype], seed=N + K, bias=bias)
    g = torch.Generator(device="cuda").manual_seed(5)
    up = [torch.randn(B, N, generator=g, device="cuda") * v for v in (1.0, 0.1, 0.3)]
    if bias == "mask":  # a masked target's logp is -inf: weigh only those that are not
        hit = b.gather(1, ids.clamp(min=0).long()) == -math.inf
        up[0][hit] = 0.0
    leaves = [t.requires_grad_(True) for t in (x, c, b) if t is not None]
    r = token_log_probs(x, c, ids, scale=0.7, bias=b)
    got = torch.autograd.grad([r.logp, r.lse, r.entropy], leaves, up)
    with torch.no_grad():
        want, absG, tol = reference_grads(x, c, ids, 0.7, b, up)
        T = TYPES[dtype]
        step = torch.finfo(T).eps / 2
        # G held as three bf16 parts (fp32): 2^-25 of each value
        ground = 2.0 ** -25 if dtype == "fp32" else step
        pairs = 6 if dtype == "fp32" else 1
        # a score error tol_n changes p by the factor 1 + 2 tol_n and log p by 2 tol_n
        eG = absG * (4 * tol * (1 + math.log(K))).unsqueeze(-1)
        for i, (a, w) in enumerate(zip(got, want)):
            if i == 2:  # column sums before the rounding: fp32 sums of N terms
                bound = eG.sum(1) + absG.sum(1) * (N / 32 + 8) * U
                assert ((a - w).abs() <= bound + 1e-30).all(), "dbias"
                continue
            other = (c if i == 0 else x).detach().double().abs()
            M = absG if i == 0 else absG.transpose(1, 2)
            E = eG if i == 0 else eG.transpose(1, 2)
            n = M.shape[-1]
            lin = 0.7 * (M @ other) * (ground + ((n / 16 + 20) * pairs + 4) * U)
            bound = lin + 0.7 * (E @ other) + w.abs() * step
            if dtype == "fp16":  # subnormal results, and subnormal entries of the scaled G (bound / 2^13 / 2^25)
                big = absG.sum(-1).amax() * 4 + 1
                bound = bound + 2.0 ** -25 + 0.7 * big * 2.0 ** -38 * other.sum(1, keepdim=True)
            assert ((a.double() - w).abs() <= bound).all(), ("dx", "dc")[i]
    assert fk.fk_device_error() == fk.FK_OK
