"""Measured cases of the soft assignment operators: token log probabilities and the mixture-of-experts layer.

``run`` computes an operator either in its plain form (elementary torch operations in
32 bits) or, where ``own`` is true, through the framework's public calls.

Three kinds of case:

- ``score``: log probabilities of given ids against a table of K vectors, with the
  log normaliser, the entropy and the ``top`` likeliest alternatives;
- ``train``: the same with the gradients of rows, table (and bias) for given upstream
  gradients;
- ``moe``: a mixture-of-experts layer for a few tokens.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def _score(name, B, N, K, d, dtype, top, bias=False):
    return {"name": name, "kind": "score", "B": B, "N": N, "K": K, "d": d, "dtype": dtype, "top": top, "bias": bias}


def _train(name, N, K, d, dtype, entropy=False, bias=False):
    return {"name": name, "kind": "train", "B": 1, "N": N, "K": K, "d": d, "dtype": dtype, "top": 0, "bias": bias,
            "entropy": entropy}


def _moe(name, T, E, k, d, F, dtype, renorm=True):
    return {"name": name, "kind": "moe", "T": T, "E": E, "k": k, "d": d, "F": F, "dtype": dtype, "renorm": renorm}


def listed():
    return [
        # one decoded token with its alternatives: the table is read once, latency counts
        _score("one row", 1, 1, 32000, 2048, "bf16", 8),
        # a decode step of a small batch against a large vocabulary
        _score("decode batch", 1, 16, 131072, 4096, "fp16", 5),
        # scoring a ragged prompt: odd row count, odd vocabulary
        _score("prompt scoring", 1, 1999, 50021, 1024, "bf16", 4),
        # soft assignment of the API benchmark's point sets (8 of its batches) to 1000 centroids: bias = -|c|^2
        _score("soft assignment", 8, 75600, 1000, 128, "fp16", 2, bias=True),
        # a reference evaluation in full precision
        _score("fp32 scoring", 1, 1000, 8191, 512, "fp32", 3),
        # a small head over cluster ids
        _train("small codebook head", 512, 1000, 256, "bf16"),
        # a pretraining micro-batch
        _train("vocabulary head", 4096, 65536, 2048, "bf16"),
        # a policy step: weighted rows, entropy and normaliser terms, biased head
        _train("policy head", 1777, 20003, 1024, "fp16", entropy=True, bias=True),
        # the same in full precision
        _train("fp32 head", 1024, 4099, 256, "fp32", entropy=True),
        # one decoded token through many small experts
        _moe("one token", 1, 64, 8, 2048, 1024, "bf16"),
        # a decode batch over few large experts
        _moe("few large experts", 8, 8, 2, 4096, 4096, "fp16"),
        # the largest: nearly every expert is hit
        _moe("many small experts", 64, 128, 8, 2048, 768, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["score", "train", "moe"])
    if kind == "moe":
        while True:
            T, d, F = _log_int(rng, 1, 128), 8 * _log_int(rng, 16, 512), 8 * _log_int(rng, 16, 512)
            E = _log_int(rng, 4, 256)
            k = rng.randint(1, min(8, E))
            # no more weights than the largest listed case, nor more products than its tokens make
            if E * d * F <= 128 * 2048 * 768 and T * k * d * F <= 64 * 8 * 2048 * 768:
                break
        return {"kind": "moe", "T": T, "E": E, "k": k, "d": d, "F": F, "dtype": rng.choice(["bf16", "fp16"]),
                "renorm": rng.random() < 0.5}
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp16", "fp32"])
    while True:
        B = rng.choice([1, 1, 1, rng.randint(2, 8)]) if kind == "score" else 1
        N, K = _log_int(rng, 1, 8192), _log_int(rng, 16, 131072)
        d = _log_int(rng, 16, 4096) if dtype == "fp32" else 8 * _log_int(rng, 2, 512)
        # at most a quarter of the largest listed case's products in full precision
        if B * N * K * d <= 4096 * 65536 * 2048 // (8 if dtype == "fp32" else 1) and B * N * K <= 1 << 28:
            break
    case = {"kind": kind, "B": B, "N": N, "K": K, "d": d, "dtype": dtype, "top": 0, "bias": rng.random() < 0.3}
    if kind == "score":
        case["top"] = min(K, rng.randint(0, 8))
    else:
        case["entropy"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["kind"] == "moe":
        T, E, d, F = case["T"], case["E"], case["d"], case["F"]
        s = dict(case)
        s["x"] = normal(T, d).to(dt)
        s["router"] = (normal(E, d) * (1.5 / math.sqrt(d))).to(dt)
        s["w_in"] = torch.empty(E, 2 * F, d, device="cuda", dtype=dt).normal_(0.0, 1 / math.sqrt(d), generator=g)
        s["w_out"] = torch.empty(E, d, F, device="cuda", dtype=dt).normal_(0.0, 1 / math.sqrt(F), generator=g)
        return s
    B, N, K, d = case["B"], case["N"], case["K"], case["d"]
    s = dict(case)
    s["ids"] = torch.randint(0, K, (B, N), generator=g, device="cuda", dtype=torch.int32)
    c = normal(B, K, d) * (2.5 / math.sqrt(d))
    # rows lean to their own token's vector, as a trained model's do
    x = normal(B, N, d)
    for b in range(B):
        x[b] += c[b][s["ids"][b].long()]
    if N > 4:
        # padding: rows whose token is ignored
        s["ids"][:, N - N // 5:] = -1
    s["scale"], s["b"] = 1.0, None
    if case["bias"] and case["kind"] == "score":
        # squared distance at temperature: -(|x|^2) / 2 is the same for every entry of a row and drops out
        s["b"] = -0.5 * c.to(dt).float().square().sum(-1)
    elif case["bias"]:
        s["b"] = normal(B, K)
    s["x"], s["c"] = x.to(dt), c.to(dt)
    if case["kind"] == "train":
        for t in ("x", "c", "b"):
            if s[t] is not None:
                s[t].requires_grad_(True)
        # a loss summed over rows: weights of a policy gradient, or plain cross entropy
        if case["entropy"]:
            s["dlogp"], s["dlse"], s["dentropy"] = -normal(B, N), normal(B, N) * 1e-2, normal(B, N) * 1e-2
        else:
            s["dlogp"] = torch.full((B, N), -1.0, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    if s["kind"] == "moe":
        return _plain_moe(s)
    with torch.no_grad():
        return _plain_score(s) if s["kind"] == "score" else _plain_train(s)


def _run_own(s):
    from clustering_flashassign_b200 import soft

    if s["kind"] == "moe":
        r = soft.expert_mixture(s["x"], s["router"], s["w_in"], s["w_out"], s["k"], renormalize=s["renorm"])
        return {"y": r.y, "expert_ids": r.expert_ids, "expert_weights": r.expert_weights}
    r = soft.token_log_probs(s["x"], s["c"], s["ids"], scale=s["scale"], bias=s["b"], top=s["top"])
    out = {"logp": r.logp, "lse": r.lse, "entropy": r.entropy}
    if s["kind"] == "score":
        if s["top"]:
            out["top_ids"], out["top_logp"] = r.top_ids, r.top_logp
        return out
    names = [n for n in ("x", "c", "b") if s[n] is not None]
    outs, ups = [r.logp], [s["dlogp"]]
    if s["entropy"]:
        outs, ups = [r.logp, r.lse, r.entropy], [s["dlogp"], s["dlse"], s["dentropy"]]
    grads = torch.autograd.grad(outs, [s[n] for n in names], ups)
    out = {n: v.detach() for n, v in out.items()}
    out.update({"d" + n: v for n, v in zip(names, grads)})
    return out


def _plain_stats(s):
    """Scores (B, N, K) in 32 bits, their probabilities, and each row's outputs."""
    scores = (s["x"].float() @ s["c"].float().transpose(1, 2)) * s["scale"]
    if s["b"] is not None:
        scores = scores + s["b"].unsqueeze(1)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - m)
    z = p.sum(-1, keepdim=True)
    lse = m + torch.log(z)
    p = p / z
    valid = s["ids"] >= 0
    at = s["ids"].clamp(min=0).long().unsqueeze(-1)
    logp = torch.where(valid, (scores.gather(-1, at) - lse).squeeze(-1), 0.0)
    entropy = -(p * (scores - lse)).sum(-1)
    return scores, p, valid, at, {"logp": logp, "lse": lse.squeeze(-1), "entropy": entropy}


def _plain_score(s):
    scores, _, _, _, out = _plain_stats(s)
    top = s["top"]
    if top:
        # neighbours in rank can lie closer than 32 bits tell apart: the order is settled in 64
        B, N, K = scores.shape
        cand = torch.topk(scores, min(K, top + 4), dim=-1).indices.sort(-1).values
        row = torch.arange(B, device="cuda").view(B, 1, 1).expand_as(cand)
        near = (s["x"].double().unsqueeze(2) * s["c"].double()[row, cand]).sum(-1) * s["scale"]
        if s["b"] is not None:
            near = near + s["b"].double()[row, cand]
        near, order = near.sort(dim=-1, descending=True, stable=True)
        out["top_ids"] = cand.gather(-1, order)[..., :top].int()
        out["top_logp"] = (near[..., :top] - out["lse"].unsqueeze(-1)).float()
    return out


def _plain_train(s):
    scores, p, valid, at, out = _plain_stats(s)
    a = torch.where(valid, s["dlogp"], 0.0).unsqueeze(-1)
    if s["entropy"]:
        lse, ent = out["lse"].unsqueeze(-1), out["entropy"].unsqueeze(-1)
        grad = p * (s["dlse"].unsqueeze(-1) - a - s["dentropy"].unsqueeze(-1) * (scores - lse + ent))
    else:
        grad = p * -a
    grad.scatter_add_(-1, at, a)
    out["dx"] = ((grad @ s["c"].float()) * s["scale"]).to(s["x"].dtype)
    out["dc"] = ((grad.transpose(1, 2) @ s["x"].float()) * s["scale"]).to(s["c"].dtype)
    if s["b"] is not None:
        out["db"] = grad.sum(1)
    return out


def _plain_moe(s):
    x, k, E, F = s["x"].float(), s["k"], s["E"], s["F"]
    T = x.shape[0]
    # which experts are chosen can hang on the last bits of two scores: 64 bits
    scores = s["x"].double() @ s["router"].double().T
    order = scores.sort(dim=-1, descending=True, stable=True)
    ids = order.indices[:, :k]
    p = torch.exp(scores - order.values[:, :1])
    w = p.gather(1, ids) / (p.gather(1, ids) if s["renorm"] else p).sum(-1, keepdim=True)
    w = w.float()
    if T * k <= E:  # few rows: only the chosen experts' weights
        h = (s["w_in"][ids].float() @ x.view(T, 1, -1, 1)).squeeze(-1)  # (T, k, 2F)
        h = h[..., :F] / (1 + torch.exp(-h[..., :F])) * h[..., F:]
        y = ((s["w_out"][ids].float() @ h.unsqueeze(-1)).squeeze(-1) * w.unsqueeze(-1)).sum(1)
    else:  # every expert, and the weights of those not chosen are zero
        h = x.unsqueeze(0) @ s["w_in"].float().transpose(1, 2)  # (E, T, 2F)
        h = h[..., :F] / (1 + torch.exp(-h[..., :F])) * h[..., F:]
        dense = torch.zeros(T, E, device="cuda").scatter_(1, ids, w)
        y = ((h * dense.T.unsqueeze(-1)) @ s["w_out"].float().transpose(1, 2)).sum(0)
    return {"y": y.to(s["x"].dtype), "expert_ids": ids.int(), "expert_weights": w}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["kind"] == "moe":
        T, E, k, d, F = (case[n] for n in ("T", "E", "k", "d", "F"))
        hit = E * (1 - (1 - k / E) ** T)  # experts that some token chooses, were the choices even
        return {"bytes": int(3 * hit * F * d * e + E * d * e + 2 * T * d * e + 8 * T * k),
                "flops": int(6 * T * k * F * d + 2 * T * E * d)}
    B, N, K, d = (case[n] for n in ("B", "N", "K", "d"))
    tables = B * (N + K) * d * e + (4 * B * K if case["bias"] else 0)
    rows = B * N * (16 + 8 * case["top"])
    if case["kind"] == "score":
        return {"bytes": tables + rows, "flops": 2 * B * N * K * d}
    return {"bytes": 2 * tables + rows + B * N * (12 if case["entropy"] else 4), "flops": 6 * B * N * K * d}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return _exact_moe(s) if s["kind"] == "moe" else _exact_rows(s)


def _exact_rows(s):
    keys = ["logp", "lse", "entropy"]
    if s["kind"] == "train":
        keys += ["dx", "dc"] + (["db"] if s["b"] is not None else [])
    elif s["top"]:
        keys += ["top_logp"]
    out = {n: [] for n in keys}
    for b in range(s["B"]):
        x, c, ids = s["x"][b].double(), s["c"][b].double(), s["ids"][b].long()
        z = torch.einsum("nd,kd->nk", x, c).mul_(s["scale"])
        if s["b"] is not None:
            z += s["b"][b].double()
        out["lse"].append(torch.logsumexp(z, 1))
        z -= out["lse"][-1][:, None]  # log probabilities
        keep = (ids >= 0).double()
        row = torch.arange(len(ids), device="cuda")
        out["logp"].append(z[row, ids.clamp(min=0)] * keep)
        out["entropy"].append(torch.special.entr(z.exp()).sum(1))
        if s["kind"] == "score":
            if s["top"]:
                out["top_logp"].append(torch.topk(z, s["top"], dim=1).values)
            continue
        a = s["dlogp"][b].double() * keep
        hot = torch.zeros_like(z)
        hot[row, ids.clamp(min=0)] = keep
        q = z.exp()
        up = a[:, None] * (hot - q)
        if s["entropy"]:
            up += s["dlse"][b].double()[:, None] * q
            up -= s["dentropy"][b].double()[:, None] * q * (z + out["entropy"][-1][:, None])
        out["dx"].append(torch.einsum("nk,kd->nd", up, c) * s["scale"])
        out["dc"].append(torch.einsum("nk,nd->kd", up, x) * s["scale"])
        if s["b"] is not None:
            out["db"].append(up.sum(0))
    out = {n: torch.stack(v) for n, v in out.items()}
    if s["kind"] == "score" and s["top"]:
        out["top_ids"] = None
    return out


def _exact_moe(s):
    x, F = s["x"].double(), s["F"]
    probs = torch.softmax(torch.einsum("td,ed->te", x, s["router"].double()), 1)
    best = torch.topk(probs, s["k"], dim=1)
    w = best.values / best.values.sum(1, keepdim=True) if s["renorm"] else best.values
    y = torch.zeros_like(x)
    for e in range(s["E"]):
        t, j = torch.nonzero(best.indices == e, as_tuple=True)
        if len(t):
            up = torch.einsum("td,fd->tf", x[t], s["w_in"][e].double())
            mid = torch.nn.functional.silu(up[:, :F]) * up[:, F:]
            y.index_add_(0, t, torch.einsum("tf,df->td", mid, s["w_out"][e].double()) * w[t, j][:, None])
    return {"y": y, "expert_ids": None, "expert_weights": w}
