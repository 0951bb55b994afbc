"""The soft assignment operators as a program uses them: masks and non-finite values,
strides, streams, captured graphs, determinism, and the operators one after another."""
import math

import pytest
import torch

import clustering_flashassign_b200 as fk
from clustering_flashassign_b200 import soft
from clustering_flashassign_b200.kmeans import FlashKMeans
from clustering_flashassign_b200.soft import expert_mixture, token_log_probs

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


def make(B, N, K, d, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randn(B, K, d, generator=g, device="cuda") * (2.5 / math.sqrt(d))
    x = torch.randn(B, N, d, generator=g, device="cuda")
    ids = torch.randint(0, K, (B, N), generator=g, device="cuda", dtype=torch.int32)
    return x.to(dtype), c.to(dtype), ids


def grads(r, leaves, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    up = [torch.randn(r.logp.shape, generator=g, device="cuda") for _ in range(3)]
    return torch.autograd.grad([r.logp, r.lse, r.entropy], leaves, up)


def same(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))


def test_masked_columns_may_hold_anything():
    x, c, ids = make(1, 70, 300, 64)
    bias = torch.zeros(1, 300, device="cuda")
    bias[:, 200:] = -INF
    bias[:, 17] = -INF
    ids[:] = ids % 200
    ids[ids == 17] = 18
    short = token_log_probs(x, c[:, :200].contiguous(), ids, bias=bias[:, :200].contiguous(), top=4)
    for junk in (NAN, INF, -INF):
        cj = c.clone()
        cj[:, 200:] = junk
        cj[:, 17] = junk
        cj.requires_grad_(True)
        xj = x.clone().requires_grad_(True)
        bj = bias.clone().requires_grad_(True)
        r = token_log_probs(xj, cj, ids, bias=bj, top=4)
        assert torch.equal(r.top_ids, short.top_ids)
        assert torch.allclose(r.logp, short.logp, atol=1e-5, rtol=0)
        assert torch.allclose(r.entropy, short.entropy, atol=1e-4, rtol=0)
        dx, dc, db = grads(r, [xj, cj, bj])
        assert all(torch.isfinite(t).all() for t in (dx, dc, db))
        assert (dc[:, 200:] == 0).all() and (dc[:, 17] == 0).all() and (db[:, 200:] == 0).all()


def test_rows_with_every_column_masked():
    x, c, ids = make(2, 40, 50, 32, torch.float16)
    bias = torch.zeros(2, 50, device="cuda")
    bias[1] = -INF
    x.requires_grad_(True), c.requires_grad_(True), bias.requires_grad_(True)
    r = token_log_probs(x, c, ids, bias=bias, top=3)
    assert (r.lse[1] == -INF).all() and (r.logp[1] == -INF).all() and (r.entropy[1] == 0).all()
    assert (r.top_ids[1] == torch.arange(3, device="cuda", dtype=torch.int32)).all() and (r.top_logp[1] == -INF).all()
    assert torch.isfinite(r.logp[0]).all()
    dx, dc, db = grads(r, [x, c, bias])
    assert (dx[1] == 0).all() and (dc[1] == 0).all() and (db[1] == 0).all()
    assert torch.isfinite(dx[0]).all() and torch.isfinite(dc[0]).all()


@pytest.mark.parametrize("N", [9, 5000])  # a block per row, a thread per row
def test_fewer_open_columns_than_alternatives(N):
    x, c, ids = make(1, N, 40, 32)
    bias = torch.full((1, 40), -INF, device="cuda")
    bias[0, [31, 5]] = 0.0
    r = token_log_probs(x, c, ids * 0 + 5, bias=bias, top=6)
    open_cols = r.top_ids[0, :, :2].sort(-1).values
    assert (open_cols == torch.tensor([5, 31], device="cuda", dtype=torch.int32)).all()
    # the masked ones follow, lowest index first
    assert (r.top_ids[0, :, 2:] == torch.tensor([0, 1, 2, 3], device="cuda", dtype=torch.int32)).all()
    assert (r.top_logp[0, :, 2:] == -INF).all()
    assert torch.isfinite(r.top_logp[0, :, :2]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_ignored_rows_and_padding_hold_anything(dtype):
    x, c, ids = make(1, 300, 500, 64, dtype)
    ids[:, 200:] = -100
    ids[:, 7] = -1
    xj = x.clone()
    xj[:, 200:] = NAN
    xj[:, 250:] = INF
    a = x.clone().requires_grad_(True)
    b = xj.requires_grad_(True)
    ca, cb = c.clone().requires_grad_(True), c.clone().requires_grad_(True)
    ra, rb = token_log_probs(a, ca, ids), token_log_probs(b, cb, ids)
    assert (ra.logp[ids < 0] == 0).all() and (rb.logp[ids < 0] == 0).all()
    assert torch.equal(ra.logp, rb.logp)
    up = torch.randn(300, device="cuda").view(1, 300)
    up[:, 200:] = NAN  # what reaches ignored rows does not count either
    ga = torch.autograd.grad([ra.logp], [a, ca], [up])
    gb = torch.autograd.grad([rb.logp], [b, cb], [up])
    assert same(ga, gb) and all(torch.isfinite(t).all() for t in gb)
    assert (gb[0][ids < 0] == 0).all()


@pytest.mark.parametrize("N", [140, 5000])
def test_nan_rows_stay_their_own(N):
    x, c, ids = make(1, N, 400, 64)
    clean = token_log_probs(x, c, ids, top=3)
    x[0, 5] = NAN
    r = token_log_probs(x, c, ids, top=3)
    assert torch.isnan(r.logp[0, 5]) and torch.isnan(r.lse[0, 5]) and torch.isnan(r.entropy[0, 5])
    assert ((r.top_ids >= 0) & (r.top_ids < 400)).all()
    keep = torch.arange(N, device="cuda") != 5
    for a, b in zip(r, clean):
        assert torch.equal(a[0, keep], b[0, keep])


def test_token_out_of_range_is_ignored_and_reported():
    x, c, ids = make(1, 10, 40, 32)
    want = token_log_probs(x, c, ids).logp
    ids[0, 3] = 40
    got = token_log_probs(x, c, ids.long() * 1).logp
    assert got[0, 3] == 0
    got[0, 3] = want[0, 3]
    assert torch.equal(got, want)
    assert fk.fk_device_error() == fk.FK_EINVAL and "token id" in fk.fk_last_error()
    assert fk.fk_device_error() == fk.FK_OK


@pytest.mark.parametrize("N", [33, 5000])
def test_ties_go_to_the_lowest_index(N):
    x, c, ids = make(1, N, 20, 32)
    table = torch.cat([c[:, torch.randperm(20)] for _ in range(60)], 1).contiguous()  # 60 copies of each row
    r = token_log_probs(x, table, ids, top=7)
    s = x.double() @ table.double().transpose(1, 2)
    want = torch.sort(s, dim=-1, descending=True, stable=True).indices[..., :7]
    assert torch.equal(r.top_ids.long(), want)


@pytest.mark.parametrize("top", [1, 2, 3, 6, 7, 10, 11, 14, 15, 28])
@pytest.mark.parametrize("N,K,d", [(3, 40, 32), (130, 3001, 64), (5000, 300, 40), (3, 900, 1032)])
def test_every_list_length(top, N, K, d):
    x, c, ids = make(1, N, K, d, seed=top)
    r = token_log_probs(x, c, ids, top=top)
    s = x.double() @ c.double().transpose(1, 2)
    want = torch.sort(s, dim=-1, descending=True, stable=True)
    assert torch.equal(r.top_ids.long(), want.indices[..., :top])
    lp = want.values[..., :top] - torch.logsumexp(s, -1, keepdim=True)
    # scores of a few units, sums of K terms: well inside 2^-23 (d / 16 + 16) sum |x c|
    assert (r.top_logp - lp).abs().max() < 2.0 ** -23 * (d / 16 + 16) * 40


def test_rising_and_falling_scores():
    """Columns in rising order beat every list again and again."""
    d, K, N = 32, 5000, 40
    c = torch.zeros(1, K, d, device="cuda", dtype=torch.float32)
    c[0, :, 0] = torch.arange(K, device="cuda") / 256
    x = torch.zeros(1, N, d, device="cuda", dtype=torch.float32)
    x[0, :, 0] = torch.linspace(-1, 1, N, device="cuda")
    ids = torch.zeros(1, N, device="cuda", dtype=torch.int32)
    for top in (2, 8, 20):
        r = token_log_probs(x, c, ids, top=top)
        s = x.double() @ c.double().transpose(1, 2)
        want = torch.sort(s, dim=-1, descending=True, stable=True).indices[..., :top]
        assert torch.equal(r.top_ids.long(), want)
        # the maximum moves by more than the slack of the running sums on the way
        assert ((r.lse - torch.logsumexp(s, -1)).abs() <= 1e-5 * (1 + s.abs().amax(-1))).all()


def test_shapes_and_strides_of_the_python_entry():
    x, c, ids = make(1, 24, 100, 64)
    want = token_log_probs(x, c, ids, top=2)
    x4 = x.view(2, 3, 4, 64)
    r = token_log_probs(x4, c[0], ids.view(2, 3, 4).long(), top=2)
    assert r.logp.shape == (2, 3, 4) and r.top_ids.shape == (2, 3, 4, 2)
    assert torch.equal(r.logp.reshape(-1), want.logp[0]) and torch.equal(r.top_ids.view(24, 2), want.top_ids[0])
    one = token_log_probs(x[0, 0], c[0], ids[0, 0], top=2)
    assert one.logp.shape == () and one.top_ids.shape == (2,)
    wide = torch.empty(1, 24, 128, device="cuda", dtype=x.dtype)
    wide[..., :64] = x
    ct = c.transpose(1, 2).contiguous().transpose(1, 2)
    assert same(token_log_probs(wide[..., :64], ct, ids, top=2), want)
    leaf = wide.clone().requires_grad_(True)
    table = c.clone().requires_grad_(True)
    g1 = grads(token_log_probs(leaf[..., :64], table, ids), [leaf, table])
    plain = x.clone().requires_grad_(True)
    t2 = c.clone().requires_grad_(True)
    g2 = grads(token_log_probs(plain, t2, ids), [plain, t2])
    assert torch.equal(g1[0][..., :64], g2[0]) and (g1[0][..., 64:] == 0).all() and torch.equal(g1[1], g2[1])
    # a shared table's gradient sums over all rows of all batches
    xb, cb, ib = make(3, 20, 50, 32, torch.float32)
    xs, cs = xb.clone().requires_grad_(True), cb[0].clone().requires_grad_(True)
    gs = torch.autograd.grad(token_log_probs(xs, cs, ib).logp.sum(), cs)[0]
    parts = []
    for b in range(3):
        cl = cb[0].clone().requires_grad_(True)
        parts.append(torch.autograd.grad(token_log_probs(xb[b], cl, ib[b]).logp.sum(), cl)[0].double())
    # fp32 sums of 60 rows against three of 20
    assert (gs.double() - sum(parts)).abs().max() <= 60 * 2.0 ** -23 * (xb.abs().amax() * 2)
    with pytest.raises(ValueError, match="contiguous"):
        o = torch.empty(1, 24, device="cuda")
        fk.fk_logprob(wide[..., :64], c, ids, o, o.clone())


def test_no_rows_and_one_column():
    x, c, ids = make(1, 4, 1, 16)
    r = token_log_probs(x, c, ids * 0, top=1)
    assert (r.top_ids == 0).all()
    # one column: p = 1.  The score is rounded once as the row's maximum and not in
    # the exponent, so log p is off by up to half a step of a base-2 score below 16
    # (2^-21), and a rounding each of the exponential and the logarithm (2^-23)
    assert (r.lse.abs() < 16 * math.log(2)).all()
    for t in (r.logp, r.top_logp, r.entropy):
        assert (t.abs() <= (2.0 ** -21 + 2 * 2.0 ** -23) * math.log(2)).all()
    assert (r.logp <= 0).all() and (r.top_logp <= 0).all() and (r.entropy >= 0).all()
    e = token_log_probs(x[:, :0], c, ids[:, :0], top=1)
    assert e.logp.shape == (1, 0) and e.top_ids.shape == (1, 0, 1)
    cl = c.clone().requires_grad_(True)
    g = torch.autograd.grad(token_log_probs(x[:, :0], cl, ids[:, :0]).logp.sum(), cl)[0]
    assert (g == 0).all()


def test_unused_gradients_are_not_computed_and_second_derivatives_refused():
    x, c, ids = make(1, 20, 60, 32)
    leaf = x.clone().requires_grad_(True)
    r = token_log_probs(leaf, c, ids)
    only = torch.autograd.grad(r.logp.sum(), leaf)[0]
    both = torch.autograd.grad(token_log_probs(leaf, c.clone().requires_grad_(True), ids).logp.sum(), leaf)[0]
    assert torch.equal(only, both)
    r = token_log_probs(leaf, c, ids)
    g = torch.autograd.grad(r.logp.sum(), leaf, create_graph=True)[0]
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.float().sum(), leaf)


def test_gradients_against_differences():
    """The loss in fp64 along random directions, by central differences."""
    x, c, ids = make(1, 30, 90, 24, torch.float32)
    ids[0, 4] = -1
    bias = torch.randn(1, 90, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    up = [torch.randn(1, 30, generator=g, device="cuda") for _ in range(3)]

    def loss(x, c, b):
        lp = torch.log_softmax(0.5 * x @ c.transpose(1, 2) + b.unsqueeze(1), -1)
        s = 0.5 * x @ c.transpose(1, 2) + b.unsqueeze(1)
        logp = lp.gather(-1, ids.clamp(min=0).long().unsqueeze(-1)).squeeze(-1) * (ids >= 0)
        ent = -(lp.exp() * lp).sum(-1)
        return sum((u.double() * v).sum() for u, v in zip(up, (logp, torch.logsumexp(s, -1), ent)))

    leaves = [t.clone().requires_grad_(True) for t in (x, c, bias)]
    r = token_log_probs(leaves[0], leaves[1], ids, scale=0.5, bias=leaves[2])
    got = torch.autograd.grad([r.logp, r.lse, r.entropy], leaves, up)
    h = 1e-5
    for i in range(3):
        for _ in range(4):
            v = torch.randn(got[i].shape, generator=g, device="cuda").double()
            at = [t.double() for t in (x, c, bias)]
            hi, lo = list(at), list(at)
            hi[i], lo[i] = at[i] + h * v, at[i] - h * v
            want = (loss(*hi) - loss(*lo)) / (2 * h)
            # differences: h^2 of a third derivative of order 1e3, 1e-16 of the loss / h; ours: fp32 sums
            norm = float((got[i].double().abs() * v.abs()).sum())
            assert abs(float((got[i].double() * v).sum() - want)) <= 1e-5 * norm + 1e-5


def test_repeats_are_bit_identical():
    x, c, ids = make(1, 700, 3001, 256, torch.float16)
    b = torch.randn(1, 3001, device="cuda")
    first = None
    for _ in range(4):
        leaves = [t.clone().requires_grad_(True) for t in (x, c, b)]
        r = token_log_probs(leaves[0], leaves[1], ids, bias=leaves[2], top=5)
        now = [t.detach() for t in r] + list(grads(r, leaves))
        assert first is None or same(first, now)
        first = now


def test_row_blocks_of_the_backward_pass():
    """Many rows against a long table: more of G than is held at a time (4 GiB)."""
    N, K, d = 40000, 60000, 32
    x, c, ids = make(1, N, K, d)
    up = torch.randn(1, N, device="cuda")
    o = torch.empty(3, 1, N, device="cuda")
    fk.fk_logprob(x, c, ids, o[0], o[1], o[2])
    dx, dc = torch.empty_like(x), torch.empty_like(c)
    fk.fk_logprob_backward(x, c, ids, o[1], dlogp=up, dx=dx, dc=dc)
    want_dx, want_dc, mass = [], torch.zeros(K, d, device="cuda", dtype=torch.float64), 0
    for n in range(0, N, 5000):
        s = x[0, n:n + 5000].float() @ c[0].float().T
        p = torch.exp(s - o[1][0, n:n + 5000, None])
        p.mul_(-up[0, n:n + 5000, None]).scatter_add_(1, ids[0, n:n + 5000, None].long(), up[0, n:n + 5000, None])
        want_dx.append(p @ c[0].float())
        want_dc += (p.T @ x[0, n:n + 5000].float()).double()
    want_dx = torch.cat(want_dx)
    # both types are rounded once (2^-9), G once more, the sums are fp32
    assert (dx[0].float() - want_dx).norm() <= 4e-3 * want_dx.norm()
    assert (dc[0].double() - want_dc).norm() <= 4e-3 * want_dc.norm()
    again = torch.empty_like(dc)
    fk.fk_logprob_backward(x, c, ids, o[1], dlogp=up, dc=again)
    assert torch.equal(dc, again)


def test_other_streams_and_two_calls_at_once():
    x, c, ids = make(1, 400, 2000, 128)
    m = [torch.randn(*s, device="cuda", dtype=torch.bfloat16) * 0.1 for s in ((16, 64), (32, 64), (32, 128, 64), (32, 64, 64))]
    want = token_log_probs(x, c, ids, top=4)
    want_m = expert_mixture(*m, 4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((token_log_probs(x, c, ids, top=4), expert_mixture(*m, 4)))
    torch.cuda.synchronize()
    for r, e in got:
        assert same(r, want) and same(e, want_m)
    # the explicit stream argument, with a workspace of the caller's (the joining
    # order, and so the last bit, depends on whether alternatives are asked for)
    want = token_log_probs(x, c, ids)
    o = torch.empty(2, 1, 400, device="cuda")
    torch.cuda.synchronize()
    fk.fk_logprob(x, c, ids, o[0], o[1], stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(o[0], want.logp)
    o.zero_()
    torch.cuda.synchronize()
    fk.fk_logprob(x, c, ids, o[0], o[1], workspace=torch.empty(1 << 24, device="cuda", dtype=torch.uint8),
                  stream=streams[1].cuda_stream)
    streams[1].synchronize()
    assert torch.equal(o[0], want.logp)


def test_captured_graphs_replay_on_new_inputs():
    x, c, ids = make(1, 200, 1500, 64)
    x2, c2, ids2 = make(1, 200, 1500, 64, seed=9)
    bias = torch.randn(1, 1500, device="cuda")
    m = [torch.randn(*s, device="cuda", dtype=torch.float16) * 0.1 for s in ((5, 64), (32, 64), (32, 128, 64), (32, 64, 64))]
    m2 = [torch.randn_like(t) * 0.1 for t in m]
    lx, lc, lb = x.clone().requires_grad_(True), c.clone().requires_grad_(True), bias.clone().requires_grad_(True)
    up = torch.randn(1, 200, device="cuda")

    def step():
        r = token_log_probs(lx, lc, ids, bias=lb, top=3)
        g = torch.autograd.grad([r.logp, r.entropy], [lx, lc, lb], [up, up])
        return [t.detach() for t in r] + list(g)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step(), expert_mixture(*m, 3)
    torch.cuda.current_stream().wait_stream(s)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        out1 = step()
    with torch.cuda.graph(g2):
        out2 = expert_mixture(*m, 3)
    big = token_log_probs(*make(1, 3000, 9000, 64), top=5)  # later, larger calls do not disturb the graphs
    for xs, cs, ms in ((x, c, m), (x2, c2, m2), (x, c, m)):
        with torch.no_grad():
            lx.copy_(xs), lc.copy_(cs)
            for a, b in zip(m, [t.clone() for t in ms]):
                a.copy_(b)
        for a in out1:
            a.zero_()
        g1.replay(), g2.replay(), g1.replay()
        torch.cuda.synchronize()
        assert same(out1, step())
        assert same(out2, expert_mixture(*m, 3))
    assert torch.isfinite(big.logp).all() and fk.fk_device_error() == fk.FK_OK


def test_fault_injection_reaches_the_soft_operators():
    x, c, ids = make(1, 8, 30, 16)
    fk.fk_inject_fault(fk.FK_FAULT_LAUNCH, 1)
    with pytest.raises(fk.FkError):
        token_log_probs(x, c, ids)
    fk.fk_inject_fault(fk.FK_FAULT_NONE)
    assert torch.isfinite(token_log_probs(x, c, ids).logp).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_clusters_soft_assignment_head_and_mixture_together(dtype):
    """Features are clustered, softly assigned, a head learns the cluster ids, and a
    mixture routed by the centroids transforms the rows."""
    g = torch.Generator(device="cuda").manual_seed(0)
    means = torch.randn(12, 64, generator=g, device="cuda") * 2
    data = (means[torch.randint(0, 12, (4000,), generator=g, device="cuda")]
            + torch.randn(4000, 64, generator=g, device="cuda")).to(dtype)
    km = FlashKMeans(d=64, k=12, niter=8, dtype=dtype)
    labels = km.fit_predict(data)
    r = km.log_prob(data, temperature=4.0, top=3)
    hard = km.predict(data)
    c = km.centroids.to(dtype)
    d2 = (data.double().unsqueeze(1) - c.double()).square().sum(-1)
    want = torch.log_softmax(-d2 / 4.0, -1)
    # -|c|^2 in fp32, scores up to a few hundred
    tol = 2.0 ** -23 * 64 * float(d2.max())
    assert (r.logp - want.gather(1, hard.long().unsqueeze(1)).squeeze(1)).abs().max() <= tol
    sure = want.topk(2, dim=1).values
    sure = (sure[:, 0] - sure[:, 1]) > 1e-2
    assert torch.equal(r.top_ids[sure, 0], hard[sure])
    asked = km.log_prob(data, ids=torch.zeros(4000, device="cuda", dtype=torch.int64), temperature=4.0)
    assert (asked.logp - want[:, 0]).abs().max() <= tol

    head = (torch.randn(12, 64, generator=g, device="cuda") * 0.1).to(dtype).requires_grad_(True)
    out = token_log_probs(data, head, labels)
    grad = torch.autograd.grad(-out.logp.mean(), head)[0]
    lp = torch.log_softmax(data.double() @ head.double().T, -1)
    ref = -(torch.nn.functional.one_hot(labels.long(), 12).double() - lp.exp()).T @ data.double() / 4000
    assert (grad.double() - ref).norm() <= 4e-3 * ref.norm()
    if dtype == torch.float16:
        w_in = (torch.randn(12, 64, 64, generator=g, device="cuda") / 8).half()
        w_out = (torch.randn(12, 64, 32, generator=g, device="cuda") / 6).half()
        e = expert_mixture(data[:20], c, w_in, w_out, 3)
        top = token_log_probs(data[:20], c, labels[:20], top=3)
        assert torch.equal(e.expert_ids, top.top_ids)
        assert torch.isfinite(e.y).all()
    assert fk.fk_device_error() == fk.FK_OK
