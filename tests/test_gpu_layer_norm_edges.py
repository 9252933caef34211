"""The layer norm on the GPU at its edges: buffers that may meet, rows whose values are equal or far from
zero."""
import numpy as np
import pytest

from tests import _recurrent_ref as ref
from tests.test_gpu_recurrence import _dtype, _np, _rand, _torch

pytestmark = pytest.mark.gpu

EPS = 1e-5
U, K = ref.U, 128 * ref.U          # K: roundings of a sum over a row, as in the reference


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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [7, 100, 264, 768, 1000, 4096, 8192, 8191, 16384])
def test_rows_of_equal_values(W, dtype, cuda_device):
    """z is 0, the output the bias, and dx is (g - mean(g)) / sqrt(eps).

    The fp32 mean of W values c is off by delta <= K|c|; the deviations are that, all the same and exact.  Their own mean is
    off by K delta, so what is left of them, times r <= 1 / sqrt(eps), is below (K + 2u) delta / sqrt(eps) =: zb.  The
    variance left is a difference of two delta^2, each within 2K + 4u: below 5K delta^2, so r is off by half that over eps.
    mean(g z) is r times a difference of two products of delta and mean(|g|), each within 2K."""
    torch, la = _torch()
    values = [1745.394, 0.1, -333.333, 1e-3, 77777.7, 1.0 / 3]
    rows = len(values)
    x = torch.tensor(values, device="cuda")[:, None].expand(rows, W).to(_dtype(dtype)).contiguous()
    c = np.abs(_np(x))[:, :1]
    rng = np.random.default_rng(W)
    w, w64 = _rand(rng, (W,), "f32")
    b, b64 = _rand(rng, (W,), "f32")
    d, d64 = _rand(rng, (rows, W), dtype)
    out, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    la.lightning_attn_layer_norm(x, out, weight=w, bias=b, eps=EPS)
    la.lightning_attn_layer_norm_backward(x, d, dx, weight=w, dweight=dw, dbias=db, eps=EPS,
                                          workspace=la.new_workspace(la.lightning_attn_layer_norm_workspace_size(rows, W)))
    delta, r = K * c, EPS ** -0.5
    zb = (K + 2 * U) * delta * r
    ref.check("out", _np(out), np.broadcast_to(b64, (rows, W)), zb * np.abs(w64) + 2 * U * np.abs(b64), dtype)
    g = d64 * w64
    mg, gabs = g.mean(1, keepdims=True), np.abs(g).mean(1, keepdims=True)
    r_rel = 2.5 * K * delta ** 2 / EPS + 8 * U
    inner_tol = K * gabs + 4 * U * (np.abs(g) + np.abs(mg)) + zb * (4 * K * r * delta + zb) * gabs
    ref.check("dx", _np(dx), r * (g - mg), r * inner_tol + r * np.abs(g - mg) * (r_rel + 4 * U), dtype)
    ref.check("dweight", _np(dw), np.zeros(W), (np.abs(d64) * zb).sum(0) * (1 + K))
    ref.check("dbias", _np(db), d64.sum(0), (rows + 16) * U * np.abs(d64).sum(0))


@pytest.mark.parametrize("W", [100, 768, 4096, 8192, 16384])
@pytest.mark.parametrize("mean", [100.0, 1e4, -3e5])
def test_rows_far_from_zero(mean, W, cuda_device):
    """fp32 rows far from zero: the output is as exact as the values themselves, not as their size's roundings.

    The first mean is off by delta <= K mean(|s|); deviations from it are rounded once, their mean is off by K times their
    size: dev_tol.  The variance: 2 |dev| dev_tol and its square, and K of the two parts of the difference."""
    torch, la = _torch()
    rows = 5
    s = (mean + torch.randn(rows, W, generator=torch.Generator().manual_seed(W))).float().cuda()
    out = torch.empty_like(s)
    la.lightning_attn_layer_norm(s, out, eps=EPS)
    s64 = _np(s)
    dev = s64 - s64.mean(1, keepdims=True)
    var = (dev * dev).mean(1, keepdims=True)
    r = 1 / np.sqrt(var + EPS)
    delta = K * np.abs(s64).mean(1, keepdims=True)
    dev_tol = (K + 3 * U) * (np.abs(dev).mean(1, keepdims=True) + delta) + 3 * U * (np.abs(dev) + delta)
    var_tol = (2 * np.abs(dev) * dev_tol + dev_tol ** 2).mean(1, keepdims=True) + 2 * K * (var + delta ** 2)
    z = dev * r
    tol = dev_tol * r + np.abs(z) * (0.5 * var_tol * r * r + 8 * U) + 2 * U * (delta * r + np.abs(z))
    ref.check("out", _np(out), z, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 150, 5000])
@pytest.mark.parametrize("W", [7, 40, 128, 200, 256, 260, 500, 512, 768, 1000, 1024, 1500, 2048, 4000, 8192, 8190, 16384])
def test_workspace_of_the_size_asked_for(W, rows, dtype, cuda_device):
    """What lies behind the workspace stays as it was, and the sums are those of a larger one."""
    torch, la = _torch()
    s, d = (torch.randn(rows, W, device="cuda").to(_dtype(dtype)) for _ in range(2))
    size = la.lightning_attn_layer_norm_workspace_size(rows, W)
    got = []
    for room in (size, size + 4096):
        buf = torch.full((size + 8192,), 0xAB, dtype=torch.uint8, device="cuda")
        dx, dw, db = torch.empty_like(s), torch.empty(W, device="cuda"), torch.empty(W, device="cuda")
        la.lightning_attn_layer_norm_backward(s, d, dx, dweight=dw, dbias=db, eps=EPS, workspace=buf[:room])
        assert (buf[size:] == 0xAB).all()
        got.append((dx, dw, db))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    with pytest.raises(la.LightningAttnError):
        la.lightning_attn_layer_norm_backward(s, d, dx, dweight=dw, eps=EPS, workspace=buf[:size - 1])
    n = (rows + 16) * U
    ref.check("dbias", _np(got[0][2]), _np(d).sum(0), n * np.abs(_np(d)).sum(0))
