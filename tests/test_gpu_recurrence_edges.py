"""The gated recurrence on the GPU where its walks differ: waits that run out in the middle of a long
walk, channel blocks walked by lone CTAs and by clusters of every size, over several tiles and rounds."""
import numpy as np
import pytest

from tests import _recurrent_ref as ref
from tests.test_gpu_recurrence import DT, _gates, _np, _rand, _torch, _ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype", DT)
def test_after_a_wait_ran_out_the_walk_ends(dtype, backward, cuda_device):
    """A CTA that sends nothing, at the begin of a walk of 12 rounds and more: its cluster waits once, not
    once a round, and sends nothing more; the other clusters' channels are as without the fault."""
    torch, la = _torch()
    rng = np.random.default_rng(3)
    T, W = 12 * 16 * 256 + 77, 200
    x, _ = _rand(rng, (1, T, W), dtype)
    f, _ = _gates(rng, (1, T, W), dtype)
    d, _ = _rand(rng, (1, T, W), dtype)
    ws, ck = _ws(la, 1, T, W, x, True), la.new_recurrence_checkpoints(T, W)
    words = ws[:256].view(torch.int32)

    def call():
        if backward:
            dx, df = torch.zeros_like(x), torch.zeros_like(x)
            la.lightning_attn_gated_recurrence_backward(x, f, d, dx, df, checkpoints=ck, workspace=ws)
            return dx, df
        out = torch.zeros_like(x)
        la.lightning_attn_gated_recurrence(x, f, out, workspace=ws)
        return out,

    la.lightning_attn_gated_recurrence(x, f, torch.empty_like(x), checkpoints=ck, workspace=ws)
    want = call()
    la.lightning_attn_check(ws)
    words[4], words[5] = 50, 2          # milliseconds, the fault
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    got = call()
    end.record()
    with pytest.raises(la.LightningAttnError) as err:
        la.lightning_attn_check(ws)
    assert err.value.status == la.LA_ERR_TIMEOUT
    assert 45 < begin.elapsed_time(end) < 300       # 12 waits would take 600
    for a, b in zip(got, want):
        assert torch.equal(a[..., 32:], b[..., 32:])        # the first cluster has at most 32 channels
    words[4:6] = 0
    for a, b in zip(call(), want):
        assert torch.equal(a, b)
    la.lightning_attn_check(ws)


@pytest.mark.parametrize("T", [0, 3, 700])
@pytest.mark.parametrize("by", [-1, 1, 3])
def test_states_that_meet(T, by, cuda_device):
    """state_out a few sequences behind or ahead of state_in in one buffer, dstate_in likewise: as apart."""
    torch, la = _torch()
    rng = np.random.default_rng(T + abs(by))
    B, W = 40, 1000
    x, f, d = _rand(rng, (B, T, W), "f32")[0], _gates(rng, (B, T, W), "f32")[0], _rand(rng, (B, T, W), "f32")[0]
    ws = _ws(la, B, B * T, W, x, True)
    buf = torch.empty(B + abs(by), W, device="cuda")
    first, last = (buf[:B], buf[by:]) if by > 0 else (buf[-by:], buf[:B])
    s = _rand(rng, (B, W), "f32")[0]
    zero = torch.zeros(B, W, device="cuda")
    for backward in (False, True):
        got = []
        for given, to in ((s, torch.empty_like(s)), (first.copy_(s), last)):
            a, b = torch.empty_like(x), torch.empty_like(x)
            if backward:
                la.lightning_attn_gated_recurrence_backward(x, f, d, a, b, zero, given, to, workspace=ws)
            else:
                la.lightning_attn_gated_recurrence(x, f, a, given, to, workspace=ws)
                b = a
            got.append((a, b, to.clone()))
        la.lightning_attn_check(ws)
        assert all(torch.equal(a, b) for a, b in zip(*got))


def _columns(W):
    """Some of W channels: the first ones, the last ones and some at the borders of blocks of 16 and 32."""
    return np.unique(np.r_[0:min(W, 20), max(0, W - 35):W, [c for c in (31, 32, 47, 48, W // 2) if c < W]])


def _walk_and_compare(la, x, f, d, s0, ds1, lens, tied, dtype, cu=None):
    """Forward with checkpoints and backward with and without them: every value written, and those of some channels held
    to the reference.  x, f, d: packed rows of `lens`, which rows behind them may follow."""
    import torch
    W, n, rows, total = x.shape[1], len(lens), sum(lens), x.shape[0]
    cols = _columns(W)
    pick = lambda t: None if t is None else _np(t[..., torch.from_numpy(cols).cuda()])  # noqa: E731
    r = ref.packed(pick(x)[:rows], pick(f)[:rows], lens, tied, pick(s0), pick(d)[:rows], pick(ds1))
    mode = la.LA_INPUT_TIED if tied else la.LA_INPUT_PLAIN
    ws, ck = _ws(la, n, total, W, x, True), la.new_recurrence_checkpoints(total, W).fill_(float("nan"))
    nan = lambda t: torch.full_like(t, float("nan"))  # noqa: E731
    shape = (n, -1, W) if cu is None else (total, W)
    view = lambda t: t.view(shape)  # noqa: E731
    out, s1 = nan(x), torch.full((n, W), float("nan"), device="cuda")
    if cu is None:
        la.lightning_attn_gated_recurrence(view(x), view(f), view(out), s0, s1, ck, mode, ws)
    else:
        la.lightning_attn_gated_recurrence_varlen(x, f, out, cu, s0, s1, ck, mode, ws)
    la.lightning_attn_check(ws)
    assert torch.isfinite(out[:rows]).all() and torch.isfinite(s1).all() and out[rows:].isnan().all()
    ref.check("out", pick(out)[:rows], r["out"], r["out_tol"], dtype)
    ref.check("state_out", pick(s1), r["state_out"], r["state_out_tol"])
    used = -(-rows // 128)
    assert torch.isfinite(ck[:used]).all()
    ref.check("checkpoints", pick(ck)[:used], r["enter"][::128], r["enter_tol"][::128])
    for saved in (ck, None):
        dx, df, ds0 = nan(x), nan(x), torch.full((n, W), float("nan"), device="cuda")
        if cu is None:
            la.lightning_attn_gated_recurrence_backward(view(x), view(f), view(d), view(dx), view(df), s0, ds1, ds0, saved,
                                                        mode, ws)
        else:
            la.lightning_attn_gated_recurrence_backward_varlen(x, f, d, dx, df, cu, s0, ds1, ds0, saved, mode, ws)
        la.lightning_attn_check(ws)
        for name, t in (("dx", dx), ("df", df)):
            assert torch.isfinite(t[:rows]).all() and t[rows:].isnan().all()
            ref.check(name, pick(t)[:rows], r[name], r[name + "_tol"], dtype)
        assert torch.isfinite(ds0).all()
        ref.check("dstate_in", pick(ds0), r["dstate_in"], r["dstate_in_tol"])


def _inputs(seed, total, n, W, dtype):
    """Drawn on the GPU: x, d normal, gates whose channels remember from 2 to about 1000 tokens, states."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    normal = lambda *shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    f = normal(total, W) + 7 * torch.rand(W, device="cuda", generator=gen)
    return normal(total, W).to(t), f.to(t), normal(total, W).to(t), normal(n, W), normal(n, W)


# Lone CTAs (more than 98 blocks of 32 channels), over 5 tiles and more: whole vectors, odd rows, several sequences.
WIDE = [(1, 1500, 3200), (2, 900, 4096), (1, 1333, 3205), (3, 700, 4104), (1, 1290, 8192), (1, 129, 3300)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("B,T,W", WIDE)
def test_wide_fixed(B, T, W, tied, dtype, cuda_device):
    torch, la = _torch()
    x, f, d, s0, ds1 = _inputs(B + T + W, B * T, B, W, dtype)
    _walk_and_compare(la, x, f, d, s0, ds1, [T] * B, tied, dtype)


# Clusters of every size that the width gives, over several rounds: 3 to 8 CTAs (blocks of 16 channels in the fp32 forward,
# of 32 otherwise), a last round that is not full.
CLUSTERS = [(1, 6100, 600), (1, 6100, 800), (1, 5000, 1001), (1, 6100, 1104), (2, 3333, 1300), (1, 6100, 1504), (1, 6100, 1600),
            (1, 6100, 2000), (3, 2000, 2303), (1, 6100, 2400), (1, 4500, 3136)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T,W", CLUSTERS)
def test_clusters_of_every_size(B, T, W, dtype, cuda_device):
    torch, la = _torch()
    x, f, d, s0, ds1 = _inputs(B + T + W, B * T, B, W, dtype)
    _walk_and_compare(la, x, f, d, s0, ds1, [T] * B, W % 16 == 0, dtype)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tied,W", [(True, 3200), (False, 3205), (False, 4096), (True, 2000), (False, 1300), (True, 1001)])
@pytest.mark.parametrize("lens", [[700, 0, 1, 333, 260, 128, 2, 0, 515], [1, 1900, 40], [5] * 300])
def test_wide_and_clusters_packed(lens, tied, W, dtype, cuda_device):
    torch, la = _torch()
    rows = sum(lens)
    x, f, d, s0, ds1 = _inputs(rows + W, rows + 90, len(lens), W, dtype)
    for t in (x, f, d):
        t[rows:] = float("nan")
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")
    _walk_and_compare(la, x, f, d, s0, ds1, lens, tied, dtype, cu)


def test_values_beyond_32_bit_offsets(cuda_device):
    """More than 2^31 values a tensor, all of them drawn: a sequence of 262300 tokens, its first and last channels held to
    the reference from the first row to the last."""
    torch, la = _torch()
    W, lens = 8192, [262300, 150]
    total = sum(lens)
    assert lens[0] * W > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(77)
    draw = lambda: torch.empty(total, W, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)  # noqa: E731
    x, d = draw(), draw()
    f = draw().add_(3.0)
    out = torch.full_like(x, float("nan"))
    s1, ds0 = (torch.full((2, W), float("nan"), device="cuda") for _ in range(2))
    ck, ws = la.new_recurrence_checkpoints(total, W), _ws(la, 2, total, W, x, True)
    cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda")
    cols = np.r_[0:3, 4100, W - 3:W]
    pick = lambda t: _np(t[:, torch.from_numpy(cols).cuda()])  # noqa: E731
    r = ref.packed(pick(x), pick(f), lens, True, None, pick(d))
    la.lightning_attn_gated_recurrence_varlen(x, f, out, cu, None, s1, ck, workspace=ws)
    ref.check("out", pick(out), r["out"], r["out_tol"], "bf16")
    ref.check("state_out", pick(s1), r["state_out"], r["state_out_tol"])
    ref.check("checkpoints", pick(ck), r["enter"][::128], r["enter_tol"][::128])
    dx, df = out.fill_(float("nan")), torch.full_like(x, float("nan"))
    la.lightning_attn_gated_recurrence_backward_varlen(x, f, d, dx, df, cu, None, None, ds0, ck, workspace=ws)
    la.lightning_attn_check(ws)
    ref.check("dx", pick(dx), r["dx"], r["dx_tol"], "bf16")
    ref.check("df", pick(df), r["df"], r["df_tol"], "bf16")
    ref.check("dstate_in", pick(ds0), r["dstate_in"], r["dstate_in_tol"])
    assert all(torch.isfinite(t[i:i + 65536]).all() for t in (dx, df) for i in range(0, total, 65536))


@pytest.mark.parametrize("B", [3, 5000])
def test_malformed_offsets_without_rows(B, cuda_device):
    """Packed batches of no rows: offsets other than zeros are reported, forward and backward; with zeros the states
    pass through, into buffers of their own, in place and shifted."""
    torch, la = _torch()
    W = 40
    x = torch.empty(0, W, device="cuda")
    e = lambda: torch.empty_like(x)  # noqa: E731
    ws = _ws(la, B, 0, W, x, True)
    zero = torch.zeros(B + 1, dtype=torch.int32, device="cuda")

    def call(backward, cu, given, to):
        if backward:
            la.lightning_attn_gated_recurrence_backward_varlen(x, x, x, e(), e(), cu, None, given, to, workspace=ws)
        else:
            la.lightning_attn_gated_recurrence_varlen(x, x, e(), cu, given, to, workspace=ws)

    for backward in (False, True):
        for at, value in ((B, 3), (1, -1), (0, 1), (2, 1)):
            cu = zero.clone()
            cu[at] = value
            call(backward, cu, None, None)
            with pytest.raises(la.LightningAttnError) as err:
                la.lightning_attn_check(ws)
            assert err.value.status == la.LA_ERR_DEVICE
        s = torch.randn(B, W, device="cuda")
        for by in (0, 1, None):
            buf = torch.empty(B + 1, W, device="cuda")
            first = buf[:B].copy_(s)
            last = torch.empty_like(s) if by is None else buf[by:by + B]
            call(backward, zero, first, last)
            assert torch.equal(last, s)
        call(backward, zero, None, last)
        assert not last.any()
        la.lightning_attn_check(ws)


@pytest.mark.parametrize("dtype,T", [("bf16", 260), ("f32", 3)])
def test_most_channels(dtype, T, cuda_device):
    """2^22 channels, the most a call takes: 131072 blocks of them, rows 8 and 16 MB apart."""
    torch, la = _torch()
    x, f, d, s0, ds1 = _inputs(T, T, 1, 1 << 22, dtype)
    _walk_and_compare(la, x, f, d, s0, ds1, [T], True, dtype)


@pytest.mark.parametrize("packed", [False, True])
def test_many_sequences(packed, cuda_device):
    """300000 sequences of one token (packed: every third is empty), forward and backward, against the formulas: with one
    token G = dout + dstate_out.  u = 2^-24: the state is a scan of one step (16u + 200u of its terms, as in the reference);
    a gate is within (8 + |f|)u and |f| < 14 here, so keep G is within 22u + u + u, and a keep G (h - x) within 44u and five
    roundings more."""
    torch, la = _torch()
    B, W = 300000, 24
    lens = np.ones(B, dtype=np.int64)
    if packed:
        lens[::3] = 0
    rows = int(lens.sum())
    x, f, d, s0, ds1 = _inputs(B, rows, B, W, "f32")
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")
    ws = _ws(la, B, rows, W, x, True)
    out, dx, df = (torch.full_like(x, float("nan")) for _ in range(3))
    s1, ds0 = (torch.full_like(s0, float("nan")) for _ in range(2))
    if packed:
        la.lightning_attn_gated_recurrence_varlen(x, f, out, cu, s0, s1, workspace=ws)
        la.lightning_attn_gated_recurrence_backward_varlen(x, f, d, dx, df, cu, s0, ds1, ds0, workspace=ws)
    else:
        v = lambda t: t.view(B, 1, W)  # noqa: E731
        la.lightning_attn_gated_recurrence(v(x), v(f), v(out), s0, s1, workspace=ws)
        la.lightning_attn_gated_recurrence_backward(v(x), v(f), v(d), v(dx), v(df), s0, ds1, ds0, workspace=ws)
    la.lightning_attn_check(ws)
    some = lens > 0
    a64, x64, d64, s64, g64 = ref.sigmoid(_np(f)), _np(x), _np(d), _np(s0)[some], _np(ds1)[some]
    keep = ref.sigmoid(-_np(f))
    h, tol = a64 * s64 + keep * x64, 216 * ref.U * (np.abs(a64 * s64) + np.abs(keep * x64))
    ref.check("out", _np(out), h, tol)
    ref.check("state_out", _np(s1)[some], h, tol)
    G, Gabs = d64 + g64, np.abs(d64) + np.abs(g64)
    ref.check("dx", _np(dx), keep * G, 32 * ref.U * keep * Gabs)
    ref.check("df", _np(df), a64 * keep * G * (s64 - x64), 64 * ref.U * a64 * keep * Gabs * (np.abs(s64) + np.abs(x64)))
    ref.check("dstate_in", _np(ds0)[some], a64 * G, 216 * ref.U * a64 * Gabs)
    assert torch.equal(s1[torch.from_numpy(~some).cuda()], s0[torch.from_numpy(~some).cuda()])
    assert torch.equal(ds0[torch.from_numpy(~some).cuda()], ds1[torch.from_numpy(~some).cuda()])
