"""The differentiable gated recurrence and layer norm on the GPU, on inputs and gradients as a program has
them: slices and parts of larger tensors that start anywhere."""
import numpy as np
import pytest

from tests import _recurrent_ref as ref
from tests.test_gpu_recurrence import DT, _gates, _np, _rand, _torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("W", [7, 100])
@pytest.mark.parametrize("packed", [False, True])
def test_recurrence_of_views(packed, W, dtype, cuda_device):
    """Inputs and states sliced off a 16-byte boundary, the outputs joined to other rows: the gradient that comes back
    starts off one too."""
    torch, la = _torch()
    from long_context_attn_b200.autograd import gated_recurrence, gated_recurrence_varlen
    rng = np.random.default_rng(W)
    lens = [70, 0, 131] if packed else [201]
    n, rows = len(lens), sum(lens)
    xs, x64 = _rand(rng, (1 + rows, W), dtype)
    fs, f64 = _gates(rng, (1 + rows, W), dtype)
    ss, s64 = _rand(rng, (1 + n, W), "f32")
    wo, wo64 = _rand(rng, (1 + rows, W), dtype)
    ws, ws64 = _rand(rng, (1 + n, W), "f32")
    for t in (xs, fs, ss):
        t.requires_grad_(True)
    x, f, s = xs[1:], fs[1:], ss[1:]
    assert W == 100 or all(t.data_ptr() % 16 for t in (x, f, s))
    if packed:
        cu = torch.tensor(np.concatenate(([-1, 0], np.cumsum(lens))), dtype=torch.int32, device="cuda")[1:]
        out, st = gated_recurrence_varlen(x, f, cu, s)
    else:
        out, st = gated_recurrence(x[None], f[None], s)
        out = out[0]
    both, state = torch.cat((xs[:1], out)), torch.cat((ss[:1], st))
    torch.autograd.backward((both, state), (wo, ws))
    r = ref.packed(x64[1:], f64[1:], lens, True, s64[1:], wo64[1:], ws64[1:])
    ref.check("out", _np(out), r["out"], r["out_tol"], dtype)
    ref.check("state_out", _np(st), r["state_out"], r["state_out_tol"])
    for t, k in ((xs, "dx"), (fs, "df"), (ss, "dstate_in")):
        ref.check(k, _np(t.grad[1:]), r[k], r[k + "_tol"], dtype if t is not ss else "f32")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("W", [7, 100])
def test_layer_norm_of_views(W, dtype, cuda_device):
    torch, la = _torch()
    from long_context_attn_b200.autograd import layer_norm
    rng = np.random.default_rng(W)
    rows = 31
    xs, x64 = _rand(rng, (1 + rows, W), dtype)
    rs, r64 = _rand(rng, (1 + rows, W), dtype)
    wb, wb64 = _rand(rng, (1 + 2 * W,), "f32")
    d, d64 = _rand(rng, (1 + rows, W), dtype)
    ds, ds64 = _rand(rng, (1 + rows, W), dtype)
    for t in (xs, rs, wb):
        t.requires_grad_(True)
    out, s = layer_norm(xs[1:], wb[1:1 + W], wb[1 + W:], residual=rs[1:])
    torch.autograd.backward((torch.cat((xs[:1], out)), torch.cat((rs[:1], s))), (d, ds))
    s64 = x64[1:] + r64[1:]
    q = ref.layer_norm(s64, wb64[1:1 + W], wb64[1 + W:], 1e-5)
    ref.check("out", _np(out), q["out"], q["out_tol"], dtype)
    q = ref.layer_norm(_np(s), wb64[1:1 + W], None, 1e-5, d64[1:], ds64[1:])
    for t in (xs, rs):
        ref.check("dx", _np(t.grad[1:]), q["dx"], q["dx_tol"], dtype)
    ref.check("dweight", _np(wb.grad[1:1 + W]), q["dweight"], q["dweight_tol"])
    ref.check("dbias", _np(wb.grad[1 + W:]), q["dbias"], q["dbias_tol"])


def test_malformed_offsets_are_found_in_the_callers_workspace(cuda_device):
    """After the forward and after the backward, each for itself; a good call then leaves the record clean."""
    torch, la = _torch()
    from long_context_attn_b200.autograd import gated_recurrence_varlen
    rows, W = 300, 64
    x = torch.randn(rows, W, device="cuda", requires_grad=True)
    ws = la.new_workspace(la.lightning_attn_gated_recurrence_workspace_size(3, rows, W, la.LA_F32, True))
    for cu, good in (([0, 200, 100, 300], False), ([0, 100, 200, 301], False), ([0, 100, 200, 300], True)):
        out, _ = gated_recurrence_varlen(x, x, torch.tensor(cu, dtype=torch.int32, device="cuda"), workspace=ws)
        for part in (lambda: None, out.sum().backward):
            part()
            if good:
                la.lightning_attn_check(ws)
                continue
            with pytest.raises(la.LightningAttnError) as err:
                la.lightning_attn_check(ws)
            assert err.value.status == la.LA_ERR_DEVICE


def _layer(torch, ag, x, r, w, b, cu):
    """Norm, then the recurrence of its two halves: outputs, and gradients by fixed weights."""
    y, s = ag.layer_norm(x, w, b, residual=r)
    u, f = y.chunk(2, -1)
    h, state = ag.gated_recurrence_varlen(u, f, cu)
    d = torch.linspace(-1, 1, h.numel(), device=h.device).view(h.shape).to(h.dtype)
    grads = torch.autograd.grad((h, s, state), (x, r, w, b), (d, torch.ones_like(s), torch.ones_like(state)))
    return [t.detach() for t in (h, state, s, *grads)]


def test_on_another_stream_and_captured(cuda_device):
    """Forward and backward on a stream of their own, and captured into a graph that is replayed on new inputs: as on the
    current stream."""
    torch, la = _torch()
    from long_context_attn_b200 import autograd as ag
    rows, W = 1500, 200
    gen = torch.Generator(device="cuda").manual_seed(3)
    data = [[torch.randn(s, device="cuda", generator=gen) for s in ((rows, W), (rows, W), (W,), (W,))] for _ in range(2)]
    cu = torch.tensor([0, 700, 700, 701, rows], dtype=torch.int32, device="cuda")
    leaf = lambda ts: [t.clone().requires_grad_(True) for t in ts]  # noqa: E731
    want = [_layer(torch, ag, *leaf(ts), cu) for ts in data]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [_layer(torch, ag, *leaf(ts), cu) for ts in data]
    side.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))
    held = leaf(data[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _layer(torch, ag, *held, cu)
    for ts, w in ((data[0], want[0]), (data[1], want[1]), (data[0], want[0])):
        with torch.no_grad():
            for t, v in zip(held, ts):
                t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
