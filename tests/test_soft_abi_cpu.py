"""CPU checks of the soft assignment entry points: bad arguments are refused on the host,
before any device work, by the C ABI and by the Python wrappers."""
import ctypes

import pytest
import torch

import clustering_flashassign_b200 as fk
from clustering_flashassign_b200 import soft

P = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1004)


def need(shape, top=0):
    n = ctypes.c_longlong(-1)
    st = fk.lib.fk_logprob_workspace(ctypes.byref(shape), top, ctypes.byref(n))
    return st, n.value


def forward(shape, x=P, c=P, bias=None, scale=1.0, ids=P, logp=P, lse=P, ent=P, top=0, ti=None, tl=None, ws=P,
            n=1 << 40):
    return fk.lib.fk_logprob(ctypes.byref(shape), x, c, bias, scale, ids, logp, lse, None, ent, top, ti, tl, ws, n,
                             None)


def backward(shape, x=P, c=P, bias=None, scale=1.0, ids=P, lse=P, ent=P, a=P, el=None, e=None, dx=P, dc=P, db=None,
             ws=P, n=1 << 40):
    return fk.lib.fk_logprob_backward(ctypes.byref(shape), x, c, bias, scale, ids, lse, None, ent, a, el, e, dx, dc, db,
                                      ws, n, None)


@pytest.mark.parametrize("B,N,K,d,dtype,status", [
    (0, 4, 8, 8, 1, fk.FK_EINVAL), (1, -1, 8, 8, 1, fk.FK_EINVAL), (1, 4, 0, 8, 1, fk.FK_EINVAL),
    (1, 4, 8, 0, 1, fk.FK_EINVAL), (1, 4, 8, 12, 1, fk.FK_EINVAL), (1, 4, 8, 12, 2, fk.FK_EINVAL),
    (1, 4, 8, 8, 7, fk.FK_EINVAL), (1, 1 << 31, 8, 8, 1, fk.FK_EINVAL), (1, (1 << 31) - 100, 8, 8, 1, fk.FK_EUNSUPPORTED),
    (1, 4, (1 << 24) + 1, 8, 1, fk.FK_EUNSUPPORTED), (70000, 4, 8, 8, 1, fk.FK_EUNSUPPORTED),
    (1, 4, 8, (1 << 20) + 8, 1, fk.FK_EUNSUPPORTED),
])
def test_shapes_are_checked(B, N, K, d, dtype, status):
    s = fk.FkShape(B, N, K, d, dtype)
    n = ctypes.c_longlong(0)
    assert need(s)[0] == status
    assert forward(s) == status
    assert fk.lib.fk_logprob_backward_workspace(ctypes.byref(s), 0, 0, ctypes.byref(n)) == status
    assert backward(s) == status


def test_more_table_rows_than_rows_and_no_rows_are_fine():
    assert need(fk.FkShape(1, 1, 1000, 8, 1))[0] == fk.FK_OK
    assert need(fk.FkShape(1, 0, 1000, 8, 1))[0] == fk.FK_OK
    assert need(fk.FkShape(1, 3, 1000, 13, 0))[0] == fk.FK_OK  # fp32 rows of any length
    n = ctypes.c_longlong(0)
    s = fk.FkShape(1, 0, 1000, 8, 1)
    assert fk.lib.fk_logprob_backward_workspace(ctypes.byref(s), 1, 1, ctypes.byref(n)) == fk.FK_OK


def test_workspace_of_large_problems_stays_bounded():
    n = ctypes.c_longlong(0)
    s = fk.FkShape(1, 1 << 20, 131072, 1024, 2)
    assert fk.lib.fk_logprob_backward_workspace(ctypes.byref(s), 0, 0, ctypes.byref(n)) == fk.FK_OK
    # 4 GiB of G, a copy of the rows, and fp32 sums of the table's gradient
    assert n.value < (4 << 30) + (1 << 20) * (1024 * 2 + 64) + 16 * 131072 * 1024 * 4 + (1 << 30)


def test_null_pointers_and_arguments():
    s = fk.FkShape(1, 4, 8, 8, 1)
    for name in ("x", "c", "ids", "logp", "lse", "ws"):
        assert forward(s, **{name: None}) == fk.FK_EINVAL, name
    for name in ("x", "c", "ids", "lse", "ws"):
        assert backward(s, **{name: None}) == fk.FK_EINVAL, name
    assert forward(s, x=ODD) == fk.FK_EINVAL and "16-byte aligned" in fk.fk_last_error()
    assert backward(s, dx=ODD) == fk.FK_EINVAL
    assert forward(s, top=9, ti=P, tl=P) == fk.FK_EINVAL  # more than K
    assert forward(fk.FkShape(1, 4, 80, 8, 1), top=29, ti=P, tl=P) == fk.FK_EINVAL
    assert forward(s, top=2) == fk.FK_EINVAL and "top_ids" in fk.fk_last_error()
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert forward(s, scale=scale) == fk.FK_EINVAL and "scale" in fk.fk_last_error()
        assert backward(s, scale=scale) == fk.FK_EINVAL
    assert forward(s, n=16) == fk.FK_EINVAL and "workspace" in fk.fk_last_error()
    assert backward(s, n=16) == fk.FK_EINVAL and "workspace" in fk.fk_last_error()
    assert backward(s, db=P) == fk.FK_EINVAL and "dbias" in fk.fk_last_error()
    assert backward(s, e=P, ent=None) == fk.FK_EINVAL and "entropy" in fk.fk_last_error()
    assert fk.lib.fk_logprob_workspace(None, 0, None) == fk.FK_EINVAL
    assert fk.lib.fk_logprob_workspace(ctypes.byref(s), 0, None) == fk.FK_EINVAL


def moe(T=2, E=4, d=16, F=8, k=2, dtype=1, act=0, ptr=P, n=1 << 40):
    s = fk.FkMoeShape(T, E, d, F, k, dtype, act, 1)
    return fk.lib.fk_moe(ctypes.byref(s), ptr, P, P, P, P, P, P, P, n, None)


@pytest.mark.parametrize("args,status", [
    (dict(T=-1), fk.FK_EINVAL), (dict(E=0), fk.FK_EINVAL), (dict(d=12), fk.FK_EINVAL), (dict(F=4), fk.FK_EINVAL),
    (dict(k=0), fk.FK_EINVAL), (dict(k=5), fk.FK_EINVAL), (dict(dtype=0), fk.FK_EUNSUPPORTED),
    (dict(dtype=9), fk.FK_EINVAL), (dict(act=2), fk.FK_EINVAL), (dict(T=257), fk.FK_EUNSUPPORTED),
    (dict(E=513), fk.FK_EUNSUPPORTED), (dict(E=40, k=17), fk.FK_EUNSUPPORTED), (dict(ptr=None), fk.FK_EINVAL),
    (dict(ptr=ODD), fk.FK_EINVAL), (dict(n=16), fk.FK_EINVAL), (dict(T=0), fk.FK_OK),
])
def test_moe_arguments_are_checked(args, status):
    assert moe(**args) == status


def test_wrappers_refuse_host_tensors_and_shapes():
    x, c = torch.zeros(1, 4, 8, dtype=torch.float16), torch.zeros(1, 6, 8, dtype=torch.float16)
    ids = torch.zeros(1, 4, dtype=torch.int32)
    o = torch.zeros(1, 4)
    with pytest.raises(ValueError, match="CUDA"):
        fk.fk_logprob(x, c, ids, o, o)
    with pytest.raises(ValueError, match="CUDA"):
        fk.fk_logprob_backward(x, c, ids, o)
    with pytest.raises(ValueError, match="CUDA"):
        soft.token_log_probs(x, c, ids)
    with pytest.raises(ValueError, match="ids"):
        soft.token_log_probs(x, c, ids[:, :3])
    with pytest.raises(ValueError, match="int32"):
        soft.token_log_probs(x, c, ids.float())
    with pytest.raises(ValueError):
        soft.token_log_probs(x[0], c, ids[0])
    w_in, w_out = torch.zeros(4, 16, 8, dtype=torch.float16), torch.zeros(4, 8, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        soft.expert_mixture(x[0], torch.zeros(4, 8, dtype=torch.float16), w_in, w_out, 2)
    with pytest.raises(ValueError, match="activation"):
        soft.expert_mixture(x[0], torch.zeros(4, 8, dtype=torch.float16), w_in, w_out, 2, activation="relu")
    with pytest.raises(RuntimeError, match="no backward"):
        soft.expert_mixture(x[0], torch.zeros(4, 8, dtype=torch.float16), w_in.requires_grad_(True), w_out, 2)
