"""The layer norm on the GPU at its edges: buffers that may meet, rows whose values are equal or far from
zero."""
import numpy as np
import pytest

from tests.test_gpu_recurrence import _torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("W", [96, 8192])
def test_sums_over_what_has_been_read(W, cuda_device):
    """dweight and dbias are written last: where weight, s or dout lie they are as in buffers of their own."""
    torch, la = _torch()
    rows = 400
    s, d = torch.randn(rows, W, device="cuda"), torch.randn(rows, W, device="cuda")
    w = torch.randn(W, device="cuda")
    ws = la.new_workspace(la.lightning_attn_layer_norm_workspace_size(rows, W))
    dx, dw, db = torch.empty_like(s), torch.empty_like(w), torch.empty_like(w)
    la.lightning_attn_layer_norm_backward(s, d, dx, weight=w, dweight=dw, dbias=db, workspace=ws)
    for k in range(3):
        s2, d2, w2, dx2, db2 = s.clone(), d.clone(), w.clone(), torch.empty_like(s), torch.empty_like(w)
        dw2 = (w2, s2[3], d2[7])[k]
        la.lightning_attn_layer_norm_backward(s2, d2, dx2, weight=w2, dweight=dw2, dbias=db2, workspace=ws)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
