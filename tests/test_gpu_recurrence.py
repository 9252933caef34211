"""The gated recurrence on the GPU against its fp64 reference, with bounds derived from the
formulas (tests/_recurrent_ref.py): shapes from one token up, odd widths, packed batches with
empty sequences and rows behind the last one, states in place, gates at their limits, streams,
captured graphs, and the two operators run together as a layer runs them."""
import numpy as np
import pytest

from tests import _recurrent_ref as ref

pytestmark = pytest.mark.gpu

DT = ["bf16", "f32"]


def _torch():
    import torch
    from long_context_attn_b200 import lightning_attn as la
    return torch, la


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _rand(rng, shape, dtype, scale=1.0):
    """A device tensor of `dtype` and the same values in fp64."""
    import torch
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(scale)).to(_dtype(dtype))
    return t.cuda(), t.double().numpy()


def _gates(rng, shape, dtype):
    """Gates whose channels remember from 2 to about 1000 tokens."""
    import torch
    t = torch.from_numpy((rng.standard_normal(shape) + rng.uniform(0, 7, shape[-1])).astype(np.float32)).to(_dtype(dtype))
    return t.cuda(), t.double().numpy()


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _ws(la, n, rows, W, x, backward=False):
    return la.new_workspace(la.lightning_attn_gated_recurrence_workspace_size(n, rows, W, la._dtype(x), backward))


# Packed batches: lengths with empty, one-token and long sequences, starts on and off the
# borders of the kernel's blocks of rows.
LENS = {
    "one": [1],
    "mixed": [5, 0, 1, 130, 0, 127, 128, 1, 1, 300, 0],
    "blocks": [256, 512, 128, 1, 255, 384],
    "many": [int(n) for n in np.random.default_rng(1).integers(0, 9, 200)],
    "long": [3, 2900, 0, 41],
    "thousands": [int(n) for n in np.random.default_rng(2).integers(0, 4, 4000)],
    "sparse": [0] * 700 + [600] + [0] * 900 + [1] + [0] * 40 + [300, 2, 0],
    "none": [0, 0, 0],
}

FIXED = [(1, 1, 64), (1, 2, 8), (3, 1, 128), (1, 127, 64), (1, 128, 64), (1, 129, 64), (2, 257, 72), (5, 100, 200),
         (1, 3000, 136), (1, 600, 1), (2, 300, 7), (1, 1025, 130), (1, 513, 1000)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("B,T,W", FIXED)
def test_fixed(B, T, W, tied, dtype, cuda_device):
    torch, la = _torch()
    rng = np.random.default_rng(B * 1000 + T + W)
    with_state = (T + W) % 2 == 0
    x, x64 = _rand(rng, (B, T, W), dtype)
    f, f64 = _gates(rng, (B, T, W), dtype)
    d, d64 = _rand(rng, (B, T, W), dtype)
    s0, s064 = _rand(rng, (B, W), "f32") if with_state else (None, None)
    ds1, ds164 = _rand(rng, (B, W), "f32") if with_state else (None, None)
    mode = la.LA_INPUT_TIED if tied else la.LA_INPUT_PLAIN
    flat = lambda a: a.reshape(B * T, W)  # noqa: E731
    r = ref.packed(flat(x64), flat(f64), [T] * B, tied, s064, flat(d64), ds164)
    out, s1 = torch.full_like(x, float("nan")), torch.full((B, W), float("nan"), device="cuda")
    ck = la.new_recurrence_checkpoints(B * T, W).fill_(float("nan"))
    ws = _ws(la, B, B * T, W, x, True)
    la.lightning_attn_gated_recurrence(x, f, out, s0, s1, ck, mode, ws)
    assert la.lightning_attn_last_path() == "recurrence"
    la.lightning_attn_check(ws)
    ref.check("out", flat(_np(out)), r["out"], r["out_tol"], dtype)
    ref.check("state_out", _np(s1), r["state_out"], r["state_out_tol"])
    ref.check("checkpoints", _np(ck), r["enter"][::128], r["enter_tol"][::128])
    got = []
    for saved in (ck, None):
        dx, df = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
        ds0 = torch.full((B, W), float("nan"), device="cuda")
        la.lightning_attn_gated_recurrence_backward(x, f, d, dx, df, s0, ds1, ds0, saved, mode, ws)
        la.lightning_attn_check(ws)
        ref.check("dx", flat(_np(dx)), r["dx"], r["dx_tol"], dtype)
        ref.check("df", flat(_np(df)), r["df"], r["df_tol"], dtype)
        ref.check("dstate_in", _np(ds0), r["dstate_in"], r["dstate_in_tol"])
        got.append((dx, df, ds0))
    for a, b in zip(*got):      # recomputed checkpoints are the same values
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tied,W", [(True, 64), (False, 24), (True, 5), (False, 200)])
@pytest.mark.parametrize("lens", sorted(LENS))
def test_packed(lens, tied, W, dtype, cuda_device):
    torch, la = _torch()
    lens = LENS[lens]
    n, rows, behind = len(lens), sum(lens), 70
    rng = np.random.default_rng(rows + W)
    total = rows + behind          # rows behind the last sequence: not read for anything, left alone
    x, x64 = _rand(rng, (total, W), dtype)
    f, f64 = _gates(rng, (total, W), dtype)
    d, d64 = _rand(rng, (total, W), dtype)
    for t in (x, f, d):
        t[rows:] = float("nan")
    s0, s064 = _rand(rng, (n, W), "f32") if W != 24 else (None, None)
    ds1, ds164 = _rand(rng, (n, W), "f32")
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")
    mode = la.LA_INPUT_TIED if tied else la.LA_INPUT_PLAIN
    r = ref.packed(x64[:rows], f64[:rows], lens, tied, s064, d64[:rows], ds164)
    out, s1 = torch.full_like(x, 7.0), torch.full((n, W), float("nan"), device="cuda")
    ck = la.new_recurrence_checkpoints(total, W)
    ws = _ws(la, n, total, W, x, True)
    la.lightning_attn_gated_recurrence_varlen(x, f, out, cu, s0, s1, ck, mode, ws)
    la.lightning_attn_check(ws)
    ref.check("out", _np(out[:rows]), r["out"], r["out_tol"], dtype)
    ref.check("state_out", _np(s1), r["state_out"], r["state_out_tol"])
    assert (out[rows:] == 7.0).all()
    for saved in (ck, None):
        dx, df = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
        ds0 = torch.full((n, W), float("nan"), device="cuda")
        la.lightning_attn_gated_recurrence_backward_varlen(x, f, d, dx, df, cu, s0, ds1, ds0, saved, mode, ws)
        la.lightning_attn_check(ws)
        ref.check("dx", _np(dx[:rows]), r["dx"], r["dx_tol"], dtype)
        ref.check("df", _np(df[:rows]), r["df"], r["df_tol"], dtype)
        ref.check("dstate_in", _np(ds0), r["dstate_in"], r["dstate_in_tol"])
        assert (dx[rows:] == 7.0).all() and (df[rows:] == 7.0).all()


@pytest.mark.parametrize("T", [5, 700])
def test_states_in_place(T, cuda_device):
    """state_out may be state_in, dstate_in may be dstate_out: the same values as apart."""
    torch, la = _torch()
    rng = np.random.default_rng(T)
    B, W = 3, 96
    x, _ = _rand(rng, (B, T, W), "bf16")
    f, _ = _gates(rng, (B, T, W), "bf16")
    d, _ = _rand(rng, (B, T, W), "bf16")
    s0, _ = _rand(rng, (B, W), "f32")
    ds1, _ = _rand(rng, (B, W), "f32")
    ws = _ws(la, B, B * T, W, x, True)
    out, s1, out2, s = torch.empty_like(x), torch.empty_like(s0), torch.empty_like(x), s0.clone()
    la.lightning_attn_gated_recurrence(x, f, out, s0, s1, workspace=ws)
    la.lightning_attn_gated_recurrence(x, f, out2, s, s, workspace=ws)
    assert torch.equal(out, out2) and torch.equal(s, s1)
    ds0, ds = torch.empty_like(ds1), ds1.clone()
    g = [torch.empty_like(x) for _ in range(4)]
    la.lightning_attn_gated_recurrence_backward(x, f, d, g[0], g[1], s0, ds1, ds0, workspace=ws)
    la.lightning_attn_gated_recurrence_backward(x, f, d, g[2], g[3], s0, ds, ds, workspace=ws)
    assert torch.equal(g[0], g[2]) and torch.equal(g[1], g[3]) and torch.equal(ds, ds0)


def test_no_tokens(cuda_device):
    torch, la = _torch()
    for packed in (False, True):
        B, W = 3, 40
        shape = (0, W) if packed else (B, 0, W)
        x = torch.empty(shape, device="cuda")
        s0, s1 = torch.randn(B, W, device="cuda"), torch.empty(B, W, device="cuda")
        cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        ws = _ws(la, B, 0, W, x, True)
        e = lambda: torch.empty_like(x)  # noqa: E731
        for given in (s0, None):
            want = s0 if given is not None else torch.zeros_like(s0)
            s1.fill_(9.0)
            if packed:
                la.lightning_attn_gated_recurrence_varlen(x, x, e(), cu, given, s1, workspace=ws)
            else:
                la.lightning_attn_gated_recurrence(x, x, e(), given, s1, workspace=ws)
            assert torch.equal(s1, want)
            s1.fill_(9.0)
            if packed:
                la.lightning_attn_gated_recurrence_backward_varlen(x, x, x, e(), e(), cu, None, given, s1, workspace=ws)
            else:
                la.lightning_attn_gated_recurrence_backward(x, x, x, e(), e(), None, given, s1, workspace=ws)
            assert torch.equal(s1, want)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,W", [(1, 64), (1, 1), (7, 5), (3, 200), (256, 1024), (65, 8192)])
def test_step(B, W, dtype, cuda_device):
    """Two steps, each against the reference from the state the step before left."""
    torch, la = _torch()
    rng = np.random.default_rng(B + W)
    state, s64 = _rand(rng, (B, W), "f32")
    for tied in (False, True):
        x, x64 = _rand(rng, (B, W), dtype)
        f, f64 = _gates(rng, (B, W), dtype)
        out = torch.empty_like(x)
        la.lightning_attn_gated_recurrence_step(x, f, out, state, la.LA_INPUT_TIED if tied else la.LA_INPUT_PLAIN)
        assert la.lightning_attn_last_path() == "recurrence-step"
        r = ref.packed(x64, f64, [1] * B, tied, s64)
        ref.check("out", _np(out), r["out"], r["out_tol"], dtype)
        ref.check("state", _np(state), r["state_out"], r["state_out_tol"])
        s64 = _np(state)


def test_steps_continue_a_prefill(cuda_device):
    """A prefill of T tokens and then one-token steps give what a prefill of all tokens gives."""
    torch, la = _torch()
    rng = np.random.default_rng(9)
    B, T, more, W = 2, 300, 4, 128
    x, x64 = _rand(rng, (B, T + more, W), "bf16")
    f, f64 = _gates(rng, (B, T + more, W), "bf16")
    r = [ref.sequence(x64[b], f64[b], True) for b in range(B)]
    state, out = torch.empty(B, W, device="cuda"), torch.empty(B, T, W, dtype=torch.bfloat16, device="cuda")
    la.lightning_attn_gated_recurrence(x[:, :T].contiguous(), f[:, :T].contiguous(), out, None, state,
                                       workspace=_ws(la, B, B * T, W, x))
    for t in range(T, T + more):
        o = torch.empty(B, W, dtype=torch.bfloat16, device="cuda")
        la.lightning_attn_gated_recurrence_step(x[:, t].contiguous(), f[:, t].contiguous(), o, state)
        for b in range(B):
            ref.check("out", _np(o[b]), r[b]["out"][t], r[b]["out_tol"][t], "bf16")


@pytest.mark.parametrize("dtype", DT)
def test_gates_at_their_limits(dtype, cuda_device):
    """f = +-inf and far beyond the range of exp: running sums, resets, and gradients that are 0."""
    torch, la = _torch()
    T, W = 400, 16
    rng = np.random.default_rng(2)
    x, x64 = _rand(rng, (1, T, W), dtype)
    pattern = np.array([np.inf, -np.inf, 200.0, -200.0, 90.0, -90.0, 0.0, 30.0])
    f64 = pattern[rng.integers(0, 8, (1, T, W))]
    f64[:, :, 0] = np.inf
    f64[:, :, 1] = -np.inf
    f = torch.from_numpy(f64).to(_dtype(dtype)).cuda()
    d, d64 = _rand(rng, (1, T, W), dtype)
    ws = _ws(la, 1, T, W, x, True)
    for tied in (False, True):
        r = ref.sequence(x64[0], _np(f)[0], tied, None, d64[0])
        out, s1, dx, df = torch.empty_like(x), torch.empty(1, W, device="cuda"), torch.empty_like(x), torch.empty_like(x)
        mode = la.LA_INPUT_TIED if tied else la.LA_INPUT_PLAIN
        la.lightning_attn_gated_recurrence(x, f, out, None, s1, None, mode, ws)
        la.lightning_attn_gated_recurrence_backward(x, f, d, dx, df, input_mode=mode, workspace=ws)
        ref.check("out", _np(out[0]), r["out"], r["out_tol"], dtype)
        ref.check("dx", _np(dx[0]), r["dx"], r["dx_tol"], dtype)
        ref.check("df", _np(df[0]), r["df"], r["df_tol"], dtype)


@pytest.mark.parametrize("what", ["x", "f", "s0", "dout", "ds1"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_channel_and_sequence(what, value, cuda_device):
    """A NaN or infinity in one channel of the middle sequence leaves everything else as it was."""
    torch, la = _torch()
    lens, W = [90, 333, 0, 1, 200], 24
    n, rows = len(lens), sum(lens)
    rng = np.random.default_rng(12)
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")
    t = dict(x=_rand(rng, (rows, W), "bf16")[0], f=_gates(rng, (rows, W), "bf16")[0], dout=_rand(rng, (rows, W), "bf16")[0],
             s0=_rand(rng, (n, W), "f32")[0], ds1=_rand(rng, (n, W), "f32")[0])
    ws = _ws(la, n, rows, W, t["x"], True)

    def run():
        out, dx, df = (torch.empty_like(t["x"]) for _ in range(3))
        s1, ds0 = torch.empty_like(t["s0"]), torch.empty_like(t["s0"])
        la.lightning_attn_gated_recurrence_varlen(t["x"], t["f"], out, cu, t["s0"], s1, workspace=ws)
        la.lightning_attn_gated_recurrence_backward_varlen(t["x"], t["f"], t["dout"], dx, df, cu, t["s0"], t["ds1"], ds0,
                                                           workspace=ws)
        return out, dx, df, s1, ds0

    clean = run()
    t[what][1 if what in ("s0", "ds1") else 90 + 150, 5] = value
    dirty = run()
    for a, b in zip(clean, dirty):
        keep = torch.ones_like(a, dtype=torch.bool)
        if a.shape[0] == rows:
            keep[90:90 + 333, 5] = False
        else:
            keep[1, 5] = False
        assert torch.equal(a[keep], b[keep])
    out, dx, df, s1, ds0 = dirty
    if what in ("x", "s0") or (what == "f" and value != value):
        assert not torch.isfinite(s1[1, 5])
    if what in ("dout", "ds1"):
        assert not torch.isfinite(ds0[1, 5]) and torch.isfinite(out.float()).all()


def test_same_call_same_bits(cuda_device):
    """Nothing depends on the order in which blocks run: 20 passes, one result."""
    torch, la = _torch()
    rng = np.random.default_rng(8)
    B, T, W = 1, 20000, 64
    x, _ = _rand(rng, (B, T, W), "f32")
    f, _ = _gates(rng, (B, T, W), "f32")
    d, _ = _rand(rng, (B, T, W), "f32")
    ws = _ws(la, B, B * T, W, x, True)
    first = None
    for _ in range(20):
        out, s1, ck = torch.empty_like(x), torch.empty(B, W, device="cuda"), la.new_recurrence_checkpoints(T, W)
        dx, df = torch.empty_like(x), torch.empty_like(x)
        la.lightning_attn_gated_recurrence(x, f, out, None, s1, ck, workspace=ws)
        la.lightning_attn_gated_recurrence_backward(x, f, d, dx, df, checkpoints=ck, workspace=ws)
        got = (out, s1, ck, dx, df)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_long_sequence(cuda_device):
    """131072 tokens of 8 channels, forward and backward, against the reference."""
    torch, la = _torch()
    rng = np.random.default_rng(21)
    T, W = 131072, 8
    x, x64 = _rand(rng, (1, T, W), "bf16")
    f, f64 = _gates(rng, (1, T, W), "bf16")
    d, d64 = _rand(rng, (1, T, W), "bf16")
    r = ref.sequence(x64[0], f64[0], True, None, d64[0])
    out, s1, dx, df = torch.empty_like(x), torch.empty(1, W, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    ck = la.new_recurrence_checkpoints(T, W)
    ws = _ws(la, 1, T, W, x, True)
    la.lightning_attn_gated_recurrence(x, f, out, None, s1, ck, workspace=ws)
    la.lightning_attn_gated_recurrence_backward(x, f, d, dx, df, checkpoints=ck, workspace=ws)
    la.lightning_attn_check(ws)
    ref.check("out", _np(out[0]), r["out"], r["out_tol"], "bf16")
    ref.check("state_out", _np(s1[0]), r["state_out"], r["state_out_tol"])
    ref.check("dx", _np(dx[0]), r["dx"], r["dx_tol"], "bf16")
    ref.check("df", _np(df[0]), r["df"], r["df_tol"], "bf16")


def test_offsets_beyond_32_bits(cuda_device):
    """More than 2^31 values a tensor: the last rows of the last channels are right (their own
    sequence, so that the reference needs no more than them)."""
    torch, la = _torch()
    W, lens = 8192, [262143, 5, 2, 300]
    total = sum(lens)
    assert total * W > 2 ** 31
    x = torch.zeros(total, W, dtype=torch.bfloat16, device="cuda")
    f = torch.zeros_like(x)
    rng = np.random.default_rng(31)
    tail = slice(lens[0], total)
    xt, x64 = _rand(rng, (sum(lens[1:]), W), "bf16")
    ft, f64 = _gates(rng, (sum(lens[1:]), W), "bf16")
    x[tail], f[tail] = xt, ft
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")
    out, s1 = torch.full_like(x, 3.0), torch.empty(4, W, device="cuda")
    ck = la.new_recurrence_checkpoints(total, W)
    ws = _ws(la, 4, total, W, x, True)
    la.lightning_attn_gated_recurrence_varlen(x, f, out, cu, None, s1, ck, workspace=ws)
    cols = np.r_[0:64, W - 64:W]
    r = ref.packed(x64[:, cols], f64[:, cols], lens[1:], True, None, x64[:, cols])
    ref.check("out", _np(out[tail])[:, cols], r["out"], r["out_tol"], "bf16")
    ref.check("state_out", _np(s1[1:])[:, cols], r["state_out"], r["state_out_tol"])
    assert not out[:lens[0]].any()
    dx, df = out, torch.full_like(x, 3.0)
    la.lightning_attn_gated_recurrence_backward_varlen(x, f, x, dx, df, cu, checkpoints=ck, workspace=ws)
    la.lightning_attn_check(ws)
    ref.check("dx", _np(dx[tail])[:, cols], r["dx"], r["dx_tol"], "bf16")
    ref.check("df", _np(df[tail])[:, cols], r["df"], r["df_tol"], "bf16")
    assert not dx[:lens[0]].any() and not df[:lens[0]].any()


def test_malformed_offsets_are_reported(cuda_device):
    """Decreasing or too large cu_seqlens: an error record, no access out of range."""
    torch, la = _torch()
    rows, W = 300, 64
    x = torch.randn(rows, W, device="cuda")
    ws = _ws(la, 3, rows, W, x, True)
    for cu in ([0, 200, 100, 300], [0, 100, 200, 301], [0, 100, 2 ** 30, 300], [0, -5, 100, 300]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        guard = torch.full((3, rows, W), 5.0, device="cuda")
        la.lightning_attn_gated_recurrence_varlen(x, x, guard[1], c, workspace=ws)
        with pytest.raises(la.LightningAttnError) as err:
            la.lightning_attn_check(ws)
        assert err.value.status == la.LA_ERR_DEVICE
        la.lightning_attn_gated_recurrence_backward_varlen(x, x, x, guard[1], torch.empty_like(x), c, workspace=ws)
        with pytest.raises(la.LightningAttnError):
            la.lightning_attn_check(ws)
        assert (guard[0] == 5.0).all() and (guard[2] == 5.0).all()
    la.lightning_attn_gated_recurrence(x[None], x[None], torch.empty_like(x)[None], workspace=ws)
    la.lightning_attn_check(ws)        # the workspace is usable again


@pytest.mark.parametrize("backward", [False, True])
def test_a_missing_sum_runs_into_the_time_limit(backward, cuda_device):
    """A CTA that sends nothing: the waits of its cluster run out after the limit that the workspace
    sets, the error is reported, the GPU stays usable and so does the workspace."""
    torch, la = _torch()
    T, W = 4096, 64
    x = torch.randn(1, T, W, device="cuda").bfloat16()
    out, dx, df = (torch.empty_like(x) for _ in range(3))
    ws = _ws(la, 1, T, W, x, True)
    ck = la.new_recurrence_checkpoints(T, W).zero_()

    def call():
        if backward:
            la.lightning_attn_gated_recurrence_backward(x, x, x, dx, df, checkpoints=ck, workspace=ws)
        else:
            la.lightning_attn_gated_recurrence(x, x, out, workspace=ws)

    words = ws[:256].view(torch.int32)
    words[4], words[5] = 50, 2          # milliseconds, the fault
    call()
    with pytest.raises(la.LightningAttnError) as err:
        la.lightning_attn_check(ws)
    assert err.value.status == la.LA_ERR_TIMEOUT
    words[4:6] = 0
    call()
    la.lightning_attn_check(ws)


def test_streams_and_graphs(cuda_device):
    """Two calls at once on two streams with a workspace each, and both captured into graphs that
    share one workspace and are replayed in turn on new inputs."""
    torch, la = _torch()
    rng = np.random.default_rng(17)
    T, W = 3000, 64
    data = []
    for _ in range(2):
        x, f, d = _rand(rng, (1, T, W), "bf16")[0], _gates(rng, (1, T, W), "bf16")[0], _rand(rng, (1, T, W), "bf16")[0]
        data.append(dict(x=x, f=f, d=d, out=torch.empty_like(x), dx=torch.empty_like(x), df=torch.empty_like(x),
                         ck=la.new_recurrence_checkpoints(T, W), ws=_ws(la, 1, T, W, x, True)))

    def call(q, ws, stream=None):
        la.lightning_attn_gated_recurrence(q["x"], q["f"], q["out"], checkpoints=q["ck"], workspace=ws, stream=stream)
        la.lightning_attn_gated_recurrence_backward(q["x"], q["f"], q["d"], q["dx"], q["df"], checkpoints=q["ck"],
                                                    workspace=ws, stream=stream)

    want = []
    for q in data:
        call(q, q["ws"])
        want.append([q[k].clone() for k in ("out", "dx", "df")])
        for k in ("out", "dx", "df"):
            q[k].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(5):
        for q, s in zip(data, streams):
            call(q, q["ws"], s)
    torch.cuda.synchronize()
    for q, w in zip(data, want):
        assert all(torch.equal(q[k], v) for k, v in zip(("out", "dx", "df"), w))
        for k in ("out", "dx", "df"):
            q[k].zero_()
    graphs = []
    for q in data:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(q, data[0]["ws"])
        graphs.append(g)
    for k in (0, 1, 1, 0):
        graphs[k].replay()
    torch.cuda.synchronize()
    for q, w in zip(data, want):
        assert all(torch.equal(q[k], v) for k, v in zip(("out", "dx", "df"), w))
    data[0]["x"].copy_(data[1]["x"])
    data[0]["f"].copy_(data[1]["f"])
    data[0]["d"].copy_(data[1]["d"])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(data[0][k], v) for k, v in zip(("out", "dx", "df"), want[1]))


def test_binding_refusals(cuda_device):
    torch, la = _torch()
    x = torch.zeros(2, 8, 64, device="cuda")
    f, out = torch.zeros_like(x), torch.empty_like(x)
    ws = _ws(la, 2, 16, 64, x, True)
    good = dict(x=x, f=f, out=out, state_in=None, state_out=None, checkpoints=None, workspace=ws)
    bad = [dict(f=f.bfloat16()), dict(f=f[:, :4]), dict(out=out.transpose(0, 1).contiguous().transpose(0, 1)),
           dict(state_in=torch.zeros(1, 64, device="cuda")), dict(state_in=torch.zeros(2, 64)),
           dict(state_out=torch.zeros(2, 64, device="cuda").bfloat16()), dict(checkpoints=torch.zeros(2, 64, device="cuda")),
           dict(workspace=ws.cpu()), dict(x=x.double(), f=f.double(), out=out.double())]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            la.lightning_attn_gated_recurrence(**{**good, **kw})
    for kw in (dict(out=x), dict(out=f), dict(workspace=None), dict(workspace=ws[:16]), dict(input_mode=2)):
        with pytest.raises(la.LightningAttnError) as err:
            la.lightning_attn_gated_recurrence(**{**good, **kw})
        assert err.value.status == la.LA_ERR_INVALID_ARG
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        la.lightning_attn_gated_recurrence_varlen(x[0], f[0], out[0], cu.long(), workspace=ws)
    with pytest.raises(ValueError):
        la.lightning_attn_gated_recurrence_varlen(x[0], f[0], out[0], cu.cpu(), workspace=ws)


@pytest.mark.parametrize("packed", [False, True])
def test_autograd_gradients(packed, cuda_device):
    """Gradients of a loss over out and the final state: against the formula's, and the whole
    loss against differences along a direction (fp64 reference)."""
    torch, la = _torch()
    from long_context_attn_b200.autograd import gated_recurrence, gated_recurrence_varlen
    rng = np.random.default_rng(40)
    lens, W = ([200, 0, 1, 156] if packed else [119, 119, 119]), 72
    n, rows = len(lens), sum(lens)
    x, x64 = _rand(rng, (rows, W), "f32")
    f, f64 = _gates(rng, (rows, W), "f32")
    s0, s064 = _rand(rng, (n, W), "f32")
    d, d64 = _rand(rng, (rows, W), "f32")
    ds, ds64 = _rand(rng, (n, W), "f32")
    for t in (x, f, s0):
        t.requires_grad_(True)
    if packed:
        cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")
        out, s1 = gated_recurrence_varlen(x, f, cu, s0)
    else:
        out, s1 = gated_recurrence(x.view(n, -1, W), f.view(n, -1, W), s0)
    ((out.reshape(rows, W) * d).sum() + (s1 * ds).sum()).backward()
    r = ref.packed(x64, f64, lens, True, s064, d64, ds64)
    for t, k in ((x, "dx"), (f, "df"), (s0, "dstate_in")):
        ref.check(k, _np(t.grad), r[k], r[k + "_tol"])

    def loss(x, f, s):
        q = ref.packed(x, f, lens, True, s)
        return (q["out"] * d64).sum() + (q["state_out"] * ds64).sum()

    step = 1e-6
    dirs = [rng.standard_normal(a.shape) for a in (x64, f64, s064)]
    up = loss(*(a + step * v for a, v in zip((x64, f64, s064), dirs)))
    down = loss(*(a - step * v for a, v in zip((x64, f64, s064), dirs)))
    grads = [_np(t.grad) for t in (x, f, s0)]
    slope = sum((g * v).sum() for g, v in zip(grads, dirs))
    # each gradient within its bound, summed along the direction; the difference quotient itself
    # is off by rounding (2^-53 of the loss's terms over the step) and by its step's square
    allowed = sum((r[k + "_tol"] + ref.HALF["f32"] * np.abs(r[k])).ravel() @ np.abs(v).ravel()
                  for k, v in zip(("dx", "df", "dstate_in"), dirs))
    size = (np.abs(r["out"] * d64)).sum() + np.abs(r["state_out"] * ds64).sum()
    assert abs(slope - (up - down) / (2 * step)) <= allowed + 1e-6 * size


def test_layer_of_norm_recurrence_and_output_transform(cuda_device):
    """As a recurrent layer runs them: residual add and norm, projections, the recurrence, the
    library's output transform; the prefill with gradients, then the same layer one token at a
    time. Every library call is held to the reference on the inputs it really got."""
    torch, la = _torch()
    from long_context_attn_b200 import autograd as ag
    torch.manual_seed(5)
    B, T, H, D = 2, 150, 4, 64
    W = H * D
    dt = torch.bfloat16
    x = torch.randn(B, T, W, device="cuda", dtype=dt)
    res = torch.randn(B, T, W, device="cuda", dtype=dt)
    wn = (1 + 0.1 * torch.randn(W, device="cuda")).requires_grad_(True)
    bn = (0.1 * torch.randn(W, device="cuda")).requires_grad_(True)
    proj = (torch.randn(W, 3 * W, device="cuda", dtype=dt) / W ** 0.5).requires_grad_(True)
    xl, rl = x.clone().requires_grad_(True), res.clone().requires_grad_(True)
    y, s = ag.layer_norm(xl, wn, bn, residual=rl)
    u, f, g = (t.contiguous() for t in (y @ proj).chunk(3, -1))
    h, state = ag.gated_recurrence(u, f)
    for t in (y, u, f, h):
        t.retain_grad()
    out = torch.empty_like(h)
    la.lightning_attn_output_transform(h.detach().view(B, T, H, D), g.detach(), out)
    d = torch.randn_like(h)
    ((h * d).sum().float() + (s * 0.5).sum().float()).backward()
    flat = lambda t: _np(t).reshape(B * T, W)  # noqa: E731
    r = ref.packed(flat(u), flat(f), [T] * B, True, None, flat(h.grad))
    ref.check("h", flat(h), r["out"], r["out_tol"], "bf16")
    ref.check("du", flat(u.grad), r["dx"], r["dx_tol"], "bf16")
    ref.check("df", flat(f.grad), r["df"], r["df_tol"], "bf16")
    s64 = flat(x) + flat(res)
    q = ref.layer_norm(s64, _np(wn), _np(bn), 1e-5)
    ref.check("y", flat(y), q["out"], q["out_tol"], "bf16")
    ref.check("s", flat(s), s64, ref.U * np.abs(s64), "bf16")
    q = ref.layer_norm(flat(s), _np(wn), None, 1e-5, flat(y.grad), np.full((B * T, W), 0.5))
    ref.check("dx", flat(xl.grad), q["dx"], q["dx_tol"], "bf16")
    assert torch.equal(xl.grad, rl.grad)
    ref.check("dweight", _np(wn.grad), q["dweight"], q["dweight_tol"])
    ref.check("dbias", _np(bn.grad), q["dbias"], q["dbias_tol"])

    # one more token for each sequence, on the state the prefill left
    state = state.detach()
    before = _np(state)
    x1, r1 = torch.randn(B, W, device="cuda", dtype=dt), torch.randn(B, W, device="cuda", dtype=dt)
    y1, s1, h1, o1 = (torch.empty_like(x1) for _ in range(4))
    la.lightning_attn_layer_norm(x1, y1, residual=r1, sum_out=s1, weight=wn.detach(), bias=bn.detach())
    u1, f1, g1 = (t.contiguous() for t in (y1 @ proj.detach()).chunk(3, -1))
    la.lightning_attn_gated_recurrence_step(u1, f1, h1, state)
    la.lightning_attn_output_transform(h1.view(B, H, D), g1, o1)
    r = ref.packed(_np(u1), _np(f1), [1] * B, True, before)
    ref.check("step", _np(h1), r["out"], r["out_tol"], "bf16")
    ref.check("state", _np(state), r["state_out"], r["state_out_tol"])
    h64, g64 = _np(h1), _np(g1)
    want = h64 / np.sqrt((h64 ** 2).mean(1, keepdims=True) + 1e-6) * ref.sigmoid(g64)
    assert np.abs(_np(o1) - want).max() <= 2e-2 * np.abs(want).max()
