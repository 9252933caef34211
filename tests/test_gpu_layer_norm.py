"""The layer norm on the GPU against its fp64 reference, with bounds derived from the formulas
(tests/_recurrent_ref.py): widths of every kind, rows from none up, residuals, rows in place,
rows with a large mean, streams and captured graphs."""
import numpy as np
import pytest

from tests import _recurrent_ref as ref
from tests.test_gpu_recurrence import _np, _rand, _torch

pytestmark = pytest.mark.gpu

EPS = 1e-5
SHAPES = [(1, 1), (3, 2), (5, 7), (1, 64), (9, 100), (300, 128), (7, 264), (33, 513), (4, 768), (130, 1000), (3, 1024),
          (5, 1032), (2, 2048), (3, 2056), (700, 4096), (2, 4100), (9, 8192), (1, 8191), (3, 12296), (2, 16384),
          (2, 16383)]


def _case(rows, W, dtype):
    """Rows as a residual stream has them: a mean and a scale of their own."""
    rng = np.random.default_rng(rows * 7 + W)
    import torch
    x, _ = _rand(rng, (rows, W), dtype)
    m, _ = _rand(rng, (rows, 1), dtype)
    x = (x.float() * (0.5 + m.float().abs()) + 3 * m.float()).to(x.dtype)
    return rng, x, _np(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,W", SHAPES)
def test_forward_and_backward(rows, W, dtype, cuda_device):
    torch, la = _torch()
    rng, x, x64 = _case(rows, W, dtype)
    res, res64 = _rand(rng, (rows, W), dtype)
    d, d64 = _rand(rng, (rows, W), dtype)
    ds, ds64 = _rand(rng, (rows, W), dtype)
    w, w64 = _rand(rng, (W,), "f32")
    b, b64 = _rand(rng, (W,), "f32")
    ws = la.new_workspace(la.lightning_attn_layer_norm_workspace_size(rows, W))
    nan = lambda *s: torch.full(s or (rows, W), float("nan"), device="cuda")  # noqa: E731
    out = nan().to(x.dtype)
    la.lightning_attn_layer_norm(x, out, weight=w, bias=b, eps=EPS)
    q = ref.layer_norm(x64, w64, b64, EPS)
    ref.check("out", _np(out), q["out"], q["out_tol"], dtype)
    la.lightning_attn_layer_norm(x, out, eps=EPS)
    q = ref.layer_norm(x64, None, None, EPS)
    ref.check("out without weight", _np(out), q["out"], q["out_tol"], dtype)
    out, s = nan().to(x.dtype), nan().to(x.dtype)
    la.lightning_attn_layer_norm(x, out, residual=res, sum_out=s, weight=w, bias=b, eps=EPS)
    s64 = x64 + res64
    ref.check("sum", _np(s), s64, ref.U * np.abs(s64), dtype)
    q = ref.layer_norm(s64, w64, b64, EPS)
    ref.check("out of the sum", _np(out), q["out"], q["out_tol"], dtype)
    for dsum, dsum64, weight, weight64 in ((None, None, w, w64), (ds, ds64, None, None)):
        dx, dw, db = nan().to(x.dtype), nan(W), nan(W)
        la.lightning_attn_layer_norm_backward(x, d, dx, dsum=dsum, weight=weight, dweight=dw, dbias=db, eps=EPS,
                                              workspace=ws)
        q = ref.layer_norm(x64, weight64, None, EPS, d64, dsum64)
        ref.check("dx", _np(dx), q["dx"], q["dx_tol"], dtype)
        ref.check("dweight", _np(dw), q["dweight"], q["dweight_tol"])
        ref.check("dbias", _np(db), q["dbias"], q["dbias_tol"])
        dx2, dw2 = torch.empty_like(dx), nan(W)
        la.lightning_attn_layer_norm_backward(x, d, dx2, dsum=dsum, weight=weight, eps=EPS)
        assert torch.equal(dx2, dx)
        la.lightning_attn_layer_norm_backward(x, d, dx2, dsum=dsum, weight=weight, dweight=dw2, eps=EPS, workspace=ws)
        assert torch.equal(dw2, dw)


@pytest.mark.parametrize("W", [200, 2048])
def test_many_rows(W, cuda_device):
    """More rows than the backward has CTAs, many times over."""
    torch, la = _torch()
    rows = 5003
    rng, x, x64 = _case(rows, W, "bf16")
    d, d64 = _rand(rng, (rows, W), "bf16")
    w, w64 = _rand(rng, (W,), "f32")
    ws = la.new_workspace(la.lightning_attn_layer_norm_workspace_size(rows, W))
    q = ref.layer_norm(x64, w64, None, EPS, d64)
    first = None
    for _ in range(3):
        dx, dw, db = torch.empty_like(x), torch.empty(W, device="cuda"), torch.empty(W, device="cuda")
        la.lightning_attn_layer_norm_backward(x, d, dx, weight=w, dweight=dw, dbias=db, eps=EPS, workspace=ws)
        first = first or (dx, dw, db)
        assert all(torch.equal(a, b) for a, b in zip(first, (dx, dw, db)))
    ref.check("dx", _np(dx), q["dx"], q["dx_tol"], "bf16")
    ref.check("dweight", _np(dw), q["dweight"], q["dweight_tol"])
    ref.check("dbias", _np(db), q["dbias"], q["dbias_tol"])


@pytest.mark.parametrize("dtype,W", [("bf16", 4096), ("f32", 520), ("f32", 7)])
def test_in_place(dtype, W, cuda_device):
    torch, la = _torch()
    rows = 11
    rng, x, _ = _case(rows, W, dtype)
    res, d, ds = (_rand(rng, (rows, W), dtype)[0] for _ in range(3))
    out, s = torch.empty_like(x), torch.empty_like(x)
    la.lightning_attn_layer_norm(x, out, residual=res, sum_out=s, eps=EPS)
    for o, k in (("x", "res"), ("res", "x"), ("new", "res"), ("x", "new")):
        t = dict(x=x.clone(), res=res.clone(), new=torch.empty_like(x))
        la.lightning_attn_layer_norm(t["x"], t[o], residual=t["res"], sum_out=t[k], eps=EPS)
        assert torch.equal(t[o], out) and torch.equal(t[k], s)
    dx = torch.empty_like(x)
    la.lightning_attn_layer_norm_backward(x, d, dx, dsum=ds, eps=EPS)
    for which in range(3):
        t = [x.clone(), d.clone(), ds.clone()]
        la.lightning_attn_layer_norm_backward(t[0], t[1], t[which], dsum=t[2], eps=EPS)
        assert torch.equal(t[which], dx)


def test_rows_of_equal_values_and_large_means(cuda_device):
    """Variance 0: the bias comes back (deviations are exact zeros), gradients stay finite; a mean
    far above the deviations costs no more than the fp32 mean's own rounding."""
    torch, la = _torch()
    W = 1000
    x = torch.full((3, W), 4.0, device="cuda")
    x[1] = 0.0
    b = torch.randn(W, device="cuda")
    out = torch.empty_like(x)
    la.lightning_attn_layer_norm(x, out, bias=b, eps=EPS)
    assert torch.equal(out, b.expand(3, W))
    dx = torch.empty_like(x)
    la.lightning_attn_layer_norm_backward(x, torch.randn_like(x), dx, eps=EPS)
    assert torch.isfinite(dx).all()
    y = 1000.0 + torch.randn(4, W, device="cuda")
    out = torch.empty_like(y)
    la.lightning_attn_layer_norm(y, out, eps=EPS)
    q = ref.layer_norm(_np(y), None, None, EPS)
    ref.check("out", _np(out), q["out"], q["out_tol"])


def test_bad_values_stay_in_their_row(cuda_device):
    torch, la = _torch()
    rows, W = 20, 256
    rng, x, _ = _case(rows, W, "bf16")
    d, _ = _rand(rng, (rows, W), "bf16")
    x2 = x.clone()
    x2[3, 7], x2[11, 200] = float("nan"), float("inf")
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[3] = keep[11] = False
    got = []
    for t in (x, x2):
        out, dx = torch.empty_like(x), torch.empty_like(x)
        la.lightning_attn_layer_norm(t, out, eps=EPS)
        la.lightning_attn_layer_norm_backward(t, d, dx, eps=EPS)
        got.append((out, dx))
    for a, b in zip(*got):
        assert torch.equal(a[keep], b[keep]) and not torch.isfinite(b[~keep].float()).any()


def test_no_rows_and_more_dimensions(cuda_device):
    torch, la = _torch()
    W = 96
    x = torch.empty(0, W, device="cuda")
    dw, db = torch.ones(W, device="cuda"), torch.ones(W, device="cuda")
    la.lightning_attn_layer_norm(x, torch.empty_like(x))
    la.lightning_attn_layer_norm_backward(x, x.clone(), torch.empty_like(x), dweight=dw, dbias=db,
                                          workspace=la.new_workspace(la.lightning_attn_layer_norm_workspace_size(0, W)))
    assert not dw.any() and not db.any()
    y = torch.randn(2, 3, 5, W, device="cuda")
    a, b = torch.empty_like(y), torch.empty(30, W, device="cuda")
    la.lightning_attn_layer_norm(y, a)
    la.lightning_attn_layer_norm(y.view(30, W), b)
    assert torch.equal(a.view(30, W), b)


def test_streams_and_graph(cuda_device):
    torch, la = _torch()
    rows, W = 700, 1024
    rng, x, _ = _case(rows, W, "bf16")
    d, _ = _rand(rng, (rows, W), "bf16")
    ws = [la.new_workspace(la.lightning_attn_layer_norm_workspace_size(rows, W)) for _ in range(2)]
    sets = [dict(out=torch.empty_like(x), dx=torch.empty_like(x), dw=torch.empty(W, device="cuda"),
                 db=torch.empty(W, device="cuda")) for _ in range(2)]

    def call(q, ws, stream=None):
        la.lightning_attn_layer_norm(x, q["out"], stream=stream)
        la.lightning_attn_layer_norm_backward(x, d, q["dx"], dweight=q["dw"], dbias=q["db"], workspace=ws, stream=stream)

    call(sets[0], ws[0])
    want = {k: v.clone() for k, v in sets[0].items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for q, w, s in zip(sets, ws, streams):
        for v in q.values():
            v.zero_()
    torch.cuda.synchronize()
    for q, w, s in zip(sets, ws, streams):
        call(q, w, s)
    torch.cuda.synchronize()
    for q in sets:
        assert all(torch.equal(q[k], want[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(sets[0], ws[0])
    for v in sets[0].values():
        v.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(sets[0][k], want[k]) for k in want)


def test_binding_refusals(cuda_device):
    torch, la = _torch()
    x = torch.zeros(4, 64, device="cuda")
    out = torch.empty_like(x)
    for kw in (dict(out=out.bfloat16()), dict(out=out[:2]), dict(residual=x[:, :32]), dict(weight=x[0].bfloat16()),
               dict(weight=x[0, :32].contiguous()), dict(bias=torch.zeros(64)), dict(x=x.t(), out=out.t())):
        with pytest.raises((ValueError, TypeError)):
            la.lightning_attn_layer_norm(**{**dict(x=x, out=out), **kw})
    for kw in (dict(eps=0.0), dict(sum_out=out)):
        with pytest.raises(la.LightningAttnError) as err:
            la.lightning_attn_layer_norm(x, out, **kw)
        assert err.value.status == la.LA_ERR_INVALID_ARG
    wide = torch.zeros(1, 16400, device="cuda")
    with pytest.raises(la.LightningAttnError) as err:
        la.lightning_attn_layer_norm(wide, torch.empty_like(wide))
    assert err.value.status == la.LA_ERR_UNSUPPORTED
    with pytest.raises(la.LightningAttnError):      # sums of weights need a workspace
        la.lightning_attn_layer_norm_backward(x, x.clone(), out, dweight=torch.empty(64, device="cuda"))


def test_autograd(cuda_device):
    torch, la = _torch()
    from long_context_attn_b200.autograd import layer_norm
    rows, W = 37, 264
    rng, x, x64 = _case(rows, W, "f32")
    res, res64 = _rand(rng, (rows, W), "f32")
    d, d64 = _rand(rng, (rows, W), "f32")
    ds, ds64 = _rand(rng, (rows, W), "f32")
    w, w64 = _rand(rng, (W,), "f32")
    b, _ = _rand(rng, (W,), "f32")
    for t in (x, res, w, b):
        t.requires_grad_(True)
    out, s = layer_norm(x, w, b, residual=res)
    ((out * d).sum() + (s * ds).sum()).backward()
    q = ref.layer_norm(_np(s), w64, None, EPS, d64, ds64)
    for t, k in ((x, "dx"), (res, "dx"), (w, "dweight"), (b, "dbias")):
        ref.check(k, _np(t.grad), q[k], q[k + "_tol"])
    # the residual broadcast by the caller: its gradient is the sum over the rows
    r1 = res.detach()[:1].clone().requires_grad_(True)
    x.grad = None
    out, s = layer_norm(x, w, b, residual=r1.expand(rows, W))
    (out * d).sum().backward()
    torch.testing.assert_close(r1.grad[0], x.grad.sum(0))
