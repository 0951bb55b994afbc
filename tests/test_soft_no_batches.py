"""Empty inputs of the soft assignment's Python entries."""
import pytest
import torch

from clustering_flashassign_b200.soft import token_log_probs

pytestmark = pytest.mark.gpu


def test_no_batches():
    x = torch.zeros(0, 5, 16, device="cuda", dtype=torch.float16).requires_grad_(True)
    c = torch.zeros(0, 7, 16, device="cuda", dtype=torch.float16).requires_grad_(True)
    b = torch.zeros(0, 7, device="cuda").requires_grad_(True)
    ids = torch.zeros(0, 5, device="cuda", dtype=torch.int32)
    r = token_log_probs(x, c, ids, bias=b, top=2)
    assert r.logp.shape == (0, 5) and r.top_ids.shape == (0, 5, 2) and r.top_logp.shape == (0, 5, 2)
    g = torch.autograd.grad(r.logp.sum(), [x, c, b])
    assert [t.shape for t in g] == [x.shape, c.shape, b.shape]


def test_no_rows_of_any_shape():
    c = torch.randn(7, 16, device="cuda", dtype=torch.float16)
    for lead in ((0,), (0, 3), (3, 0), (2, 0, 5)):
        x = torch.zeros(*lead, 16, device="cuda", dtype=torch.float16)
        table = c.clone().requires_grad_(True)
        r = token_log_probs(x, table, torch.zeros(lead, device="cuda", dtype=torch.int64), top=2)
        assert r.logp.shape == lead and r.top_ids.shape == lead + (2,)
        assert (torch.autograd.grad(r.logp.sum(), table)[0] == 0).all()
