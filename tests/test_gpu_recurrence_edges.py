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
