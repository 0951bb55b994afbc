"""Soft assignment over libfk: token log probabilities, and the experts they route to.

    r = token_log_probs(x, c, ids, top=5)
    r.logp, r.lse, r.entropy, r.top_ids, r.top_logp

    m = expert_mixture(x, router, w_in, w_out, top_k=8)
    m.y, m.expert_ids, m.expert_weights

The soft form of the hard assignment: where fk_assign picks the nearest entry of a
table for every row, this gives the log probability of a given entry (token, cluster)
under the softmax of the row's scores, with the entropy of that distribution and its
likeliest entries, without storing the scores.  It differentiates with respect to the
rows, the table and the bias.

expert_mixture sends each token to its likeliest entries of a small table (the router)
and sums what these experts make of it: the serving form of a mixture-of-experts layer.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.forward_ad import unpack_dual
from torch.autograd.function import once_differentiable

from . import (DTYPES, FK_ACT_GELU, FK_ACT_SILU, _call_logprob, _call_moe,
               fk_logprob_backward)


class TokenLogProbs(NamedTuple):
    logp: torch.Tensor                 # log probability of the given id (0 where the id is negative)
    lse: torch.Tensor                  # log of the sum of exp(score)
    entropy: torch.Tensor              # of the row's distribution
    top_ids: Optional[torch.Tensor]    # likeliest entries, int32, or None with top = 0
    top_logp: Optional[torch.Tensor]


def _refuse_tangents(where: str, *tensors) -> None:
    """Dual tensors do not require grad: without this their tangents would be dropped silently."""
    for t in tensors:
        if t is not None and unpack_dual(t).tangent is not None:
            raise RuntimeError(f"{where} has no forward-mode derivative")


def _dense(t):
    """Contiguous, and on the 16-byte border that 16-bit operands need: else a copy."""
    t = t.contiguous()
    return t.clone() if t.element_size() == 2 and t.data_ptr() % 16 else t


def _forward(x, c, bias, ids, scale, top, rest=None):
    (B, N, d), K, dev = x.shape, c.shape[1], x.device
    if not x.is_cuda or x.dtype not in DTYPES:
        raise ValueError(f"x must be an fp16, bf16 or fp32 CUDA tensor, got {x.dtype} on {dev}")
    if c.dtype != x.dtype or c.shape != (B, K, d) or c.device != dev or ids.device != dev:
        raise ValueError(f"c must be {x.dtype}, of {B} tables of width {d}, and like ids on {dev}: got {c.dtype} of "
                         f"shape {tuple(c.shape)} on {c.device}, ids on {ids.device}")
    if bias is not None and (bias.shape != (B, K) or bias.device != dev):
        raise ValueError(f"bias must be of shape {(B, K)} on {dev}: got {tuple(bias.shape)} on {bias.device}")
    logp = x.new_empty((B, N), dtype=torch.float32)
    lse, entropy = torch.empty_like(logp), torch.empty_like(logp)
    top_ids = top_logp = pi = pl = None
    if top:
        top_ids = x.new_empty((B, N, top), dtype=torch.int32)
        top_logp = x.new_empty((B, N, top), dtype=torch.float32)
        pi, pl = top_ids.data_ptr(), top_logp.data_ptr()
    if B:
        _call_logprob((B, N, K, d, DTYPES[x.dtype]), dev,
                      (x.data_ptr(), c.data_ptr(), None if bias is None else bias.data_ptr(), scale, ids.data_ptr(),
                       logp.data_ptr(), lse.data_ptr(), None if rest is None else rest.data_ptr(),
                       entropy.data_ptr(), top, pi, pl))
    return logp, lse, entropy, top_ids, top_logp


def _backward(ctx, dlogp, dlse, dentropy, *_):
    x, c, bias, ids, lse, rest, entropy = ctx.saved_tensors
    if dlogp is None and dlse is None and dentropy is None:
        return (None,) * 6
    up = [None if g is None else g.contiguous() for g in (dlogp, dlse, dentropy)]
    want = ctx.needs_input_grad
    dx = torch.empty_like(x) if want[0] else None
    dc = torch.empty_like(c) if want[1] else None
    dbias = torch.empty_like(bias) if want[2] else None
    if x.shape[0]:
        fk_logprob_backward(x, c, ids, lse, entropy, *up, dx, dc, dbias, bias, ctx.scale, lse_rest=rest)
    return dx, dc, dbias, None, None, None


_backward_once = once_differentiable(_backward)


class _LogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, c, bias, ids, scale, top):
        rest = x.new_empty(ids.shape, dtype=torch.float32)
        out = _forward(x, c, bias, ids, scale, top, rest)
        ctx.save_for_backward(x, c, bias, ids, out[1], rest, out[2])
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        if top:
            ctx.mark_non_differentiable(*out[3:])
        return out

    @staticmethod
    def backward(ctx, *grads):
        # a graph of the gradients is only recorded to refuse a second derivative
        return (_backward_once if torch.is_grad_enabled() else _backward)(ctx, *grads)


def token_log_probs(x: torch.Tensor, c: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0,
                    bias: torch.Tensor | None = None, top: int = 0) -> TokenLogProbs:
    """Log probabilities of ids under softmax(scale * x c^T + bias), with entropy and alternatives.

    x (..., d) with one table c (K, d) and ids (...), or batches x (B, N, d), c (B, K, d),
    ids (B, N); fp16, bf16 (d a multiple of 8) or fp32, x and c alike.  Strided tensors, and
    16-bit ones that start off a 16-byte border, are copied.  ids int32 or int64,
    negative: ignored (log probability 0, no gradient from it); K or more: the same, and
    fk_device_error reports it.  bias (K,) or (B, K);
    -inf masks an entry; a finite bias beyond 2.3e38 in magnitude counts as that.  top <= min(K, 28) likeliest entries, lowest index on ties
    (ordered by fp64 scores among the top + 2 largest fp32 scores).
    logp, lse and entropy are fp32 and differentiable (backward mode, once); top_ids and
    top_logp are not.
    The backward pass can be captured into a CUDA graph while no eager autograd graph of
    the same leaves is alive; fk_logprob and fk_logprob_backward can be captured always.
    """
    _refuse_tangents("token_log_probs", x, c, bias)
    if x.dim() < 1 or c.dim() not in (2, 3) or (c.dim() == 3 and x.dim() != 3):
        raise ValueError("x must be (..., d) and c (K, d), or x (B, N, d) and c (B, K, d)")
    lead = x.shape[:-1]
    if ids.shape != lead:
        raise ValueError(f"ids must be {tuple(lead)}, got {tuple(ids.shape)}")
    if ids.dtype == torch.int64:  # any value out of range stays out of range
        ids = ids.clamp(-1, c.shape[-2]).int()
    elif ids.dtype != torch.int32:
        raise ValueError(f"ids must be int32 or int64, got {ids.dtype}")
    if bias is not None and bias.dtype != torch.float32:
        bias = bias.float()
    shared = c.dim() == 2
    if shared:
        x, c, ids = x.reshape(1, -1, x.shape[-1]), c.unsqueeze(0), ids.reshape(1, -1)
        bias = None if bias is None else bias.unsqueeze(0)
    x, c, ids = _dense(x), _dense(c), ids.contiguous()
    bias = None if bias is None else bias.contiguous()
    if torch.is_grad_enabled() and (x.requires_grad or c.requires_grad or (bias is not None and bias.requires_grad)):
        out = _LogProbs.apply(x, c, bias, ids, float(scale), int(top))
    else:
        out = _forward(x, c, bias, ids, float(scale), int(top))
    if shared and (len(lead) != 2 or lead[0] != 1):
        out = [None if t is None else t.reshape(lead + t.shape[2:]) for t in out]
    return TokenLogProbs(*out)


class ExpertMixture(NamedTuple):
    y: torch.Tensor
    expert_ids: torch.Tensor       # int32, largest weight first
    expert_weights: torch.Tensor   # fp32


_ACTIVATIONS = {"silu": FK_ACT_SILU, "gelu": FK_ACT_GELU}


def expert_mixture(x: torch.Tensor, router: torch.Tensor, w_in: torch.Tensor, w_out: torch.Tensor, top_k: int, *,
                   renormalize: bool = True, activation: str = "silu") -> ExpertMixture:
    """A mixture-of-experts layer for up to 256 tokens (forward only).

    x (..., d) and router (E, d) score the experts; each token's top_k experts
    (softmax over all, lowest index on ties; renormalize: their weights sum to
    one) apply act(x gate^T) * (x up^T) with w_in (E, 2F, d), gate rows first,
    and w_out (E, d, F).  fp16 or bf16 throughout; d and F multiples of 8.  Strided
    tensors, and those that start off a 16-byte border, are copied in every call.
    It has no derivatives: inputs that require gradients, with gradients enabled,
    and dual tensors are refused.
    """
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}")
    _refuse_tangents("expert_mixture", x, router, w_in, w_out)
    if torch.is_grad_enabled() and (x.requires_grad or router.requires_grad or w_in.requires_grad
                                    or w_out.requires_grad):
        raise RuntimeError("expert_mixture has no backward pass: call it under torch.no_grad()")
    if x.dim() < 1 or router.dim() != 2 or w_in.dim() != 3 or w_out.dim() != 3:
        raise ValueError("x must be (..., d), router (E, d), w_in (E, 2F, d), w_out (E, d, F)")
    k, d, (E, _, F), dt, dev = int(top_k), x.shape[-1], w_out.shape, x.dtype, x.device
    if not x.is_cuda or dt not in DTYPES:
        raise ValueError(f"x must be an fp16 or bf16 CUDA tensor, got {dt} on {dev}")
    if (router.dtype != dt or w_in.dtype != dt or w_out.dtype != dt or router.shape != (E, d)
            or w_in.shape != (E, 2 * F, d) or w_out.shape != (E, d, F)):
        raise ValueError(f"router, w_in and w_out must be {dt} of shapes {(E, d)}, {(E, 2 * F, d)}, {(E, d, F)}: got "
                         + ", ".join(f"{t.dtype} {tuple(t.shape)}" for t in (router, w_in, w_out)))
    if router.device != dev or w_in.device != dev or w_out.device != dev:
        raise ValueError(f"x is on {dev}, the weights on {router.device}, {w_in.device}, {w_out.device}")
    flat = x.dim() == 2
    xs = _dense(x if flat else x.reshape(-1, d))
    router, w_in, w_out = _dense(router), _dense(w_in), _dense(w_out)
    T = xs.shape[0]
    y = torch.empty_like(xs)
    ids = xs.new_empty((T, k), dtype=torch.int32)
    weights = xs.new_empty((T, k), dtype=torch.float32)
    _call_moe((T, E, d, F, k, DTYPES[dt], _ACTIVATIONS[activation], int(bool(renormalize))), dev,
              (xs.data_ptr(), router.data_ptr(), w_in.data_ptr(), w_out.data_ptr(), y.data_ptr(), ids.data_ptr(),
               weights.data_ptr()))
    if flat:
        return ExpertMixture(y, ids, weights)
    lead = x.shape[:-1]
    return ExpertMixture(y.reshape(x.shape), ids.reshape(lead + (k,)), weights.reshape(lead + (k,)))
