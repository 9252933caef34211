"""The gated recurrence and the layer norm without a GPU: the fp64 references against finite
differences and closed forms, the C entries' refusals, the binding's refusals, and the autograd
functions' argument handling."""
import ctypes

import numpy as np
import pytest
import torch

from tests import _recurrent_ref as ref


@pytest.fixture(scope="module")
def lib():
    from long_context_attn_b200 import build
    return ctypes.CDLL(build.build())


# --------------------------------------------------------------------------- references
@pytest.mark.parametrize("tied", [False, True])
def test_recurrence_gradient_against_differences(tied):
    rng = np.random.default_rng(3)
    T, W = 7, 3
    x, f, dout = (rng.standard_normal((T, W)) for _ in range(3))
    s0, ds1 = rng.standard_normal((2, W))
    r = ref.sequence(x, f, tied, s0, dout, ds1)

    def loss(x, f, s0):
        q = ref.sequence(x, f, tied, s0)
        return (q["out"] * dout).sum() + (q["state_out"] * ds1).sum()

    step = 1e-6
    for name, i in (("dx", 0), ("df", 1), ("dstate_in", 2)):
        args = [x, f, s0]
        d = rng.standard_normal(args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * d, args[i] - step * d
        slope = (loss(*up) - loss(*down)) / (2 * step)
        assert abs(slope - (r[name] * d).sum()) <= 1e-7 * max(1.0, abs(slope)), name


def test_recurrence_closed_forms():
    T, W = 9, 2
    x = np.arange(1.0, T * W + 1).reshape(T, W)
    keepall = ref.sequence(x, np.full((T, W), np.inf), False)["out"]        # a = 1: running sums
    np.testing.assert_allclose(keepall, np.cumsum(x, 0))
    drop = ref.sequence(x, np.full((T, W), -np.inf), True)["out"]           # a = 0: the input itself
    np.testing.assert_allclose(drop, x)
    half = ref.sequence(np.ones((T, W)), np.zeros((T, W)), True)["out"]     # a = 1/2: 1 - 2^-t
    np.testing.assert_allclose(half[:, 0], 1 - 0.5 ** np.arange(1, T + 1))


def test_layer_norm_gradient_against_differences():
    rng = np.random.default_rng(4)
    s, dout, dsum = (rng.standard_normal((4, 6)) for _ in range(3))
    w, b = rng.standard_normal((2, 6))
    r = ref.layer_norm(s, w, b, 1e-5, dout, dsum)

    def loss(s, w, b):
        return (ref.layer_norm(s, w, b, 1e-5)["out"] * dout).sum() + (s * dsum).sum()

    step = 1e-6
    for name, i in (("dx", 0), ("dweight", 1), ("dbias", 2)):
        args = [s, w, b]
        d = rng.standard_normal(args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * d, args[i] - step * d
        slope = (loss(*up) - loss(*down)) / (2 * step)
        assert abs(slope - (r[name] * d).sum()) <= 1e-7 * max(1.0, abs(slope)), name


# --------------------------------------------------------------------------- C entries
def _ptrs(n):
    return [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(n)]


ODD = ctypes.c_void_p(0x10008)
WS = ctypes.c_void_p(0x1000000)


def test_recurrence_entries_refuse(lib):
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    fwd, var = lib.lightning_attn_gated_recurrence, lib.lightning_attn_gated_recurrence_varlen
    bwd, bvar = lib.lightning_attn_gated_recurrence_backward, lib.lightning_attn_gated_recurrence_backward_varlen
    step = lib.lightning_attn_gated_recurrence_step
    fwd.argtypes = [vp] * 6 + [i32] * 5 + [vp, sz, vp]
    var.argtypes = [vp] * 7 + [i32] * 5 + [vp, sz, vp]
    bwd.argtypes = [vp] * 9 + [i32] * 5 + [vp, sz, vp]
    bvar.argtypes = [vp] * 10 + [i32] * 5 + [vp, sz, vp]
    step.argtypes = [vp] * 4 + [i32] * 4 + [vp]
    p = _ptrs(12)

    def call(fn, packed, backward, **kw):
        a = dict(x=p[0], f=p[1], dout=p[2], out=p[3], df=p[4], s0=None, s1=None, ds1=None, ds0=None, ck=None, cu=p[5],
                 n=2, T=8, W=64, dt=1, mode=1, ws=WS, nb=1 << 40)
        a.update(kw)
        state = [a["s0"], a["ds1"], a["ds0"]] if backward else [a["s0"], a["s1"]]
        head = [a["x"], a["f"]] + ([a["dout"], a["out"], a["df"]] if backward else [a["out"]]) + state + [a["ck"]]
        return fn(*head, *([a["cu"]] if packed else []), a["n"], a["T"], a["W"], a["dt"], a["mode"], a["ws"], a["nb"],
                  None)

    for fn, packed, backward in ((fwd, 0, 0), (var, 1, 0), (bwd, 0, 1), (bvar, 1, 1)):
        bad = [dict(x=None), dict(f=None), dict(out=None), dict(x=ODD), dict(f=ODD), dict(out=ODD), dict(n=0),
               dict(T=-1), dict(W=0), dict(dt=2), dict(mode=2), dict(mode=-1), dict(s0=ODD), dict(ck=ODD),
               dict(ws=None), dict(ws=vp(0x1000010)), dict(nb=255), dict(out=p[0]), dict(out=p[1])]
        if packed:
            bad += [dict(cu=None), dict(cu=ODD)]
        if backward:
            bad += [dict(dout=None), dict(dout=ODD), dict(df=None), dict(df=ODD), dict(out=p[2]), dict(df=p[0]),
                    dict(df=p[3]), dict(ds1=ODD), dict(ds0=ODD)]
        else:
            bad += [dict(s1=ODD)]
        for kw in bad:
            assert call(fn, packed, backward, **kw) == 1, (packed, backward, kw)
    assert call(fwd, 0, 0, n=1 << 20, T=1 << 12) == 2       # 2^32 rows
    assert call(bwd, 0, 1, n=1 << 20, T=1 << 12) == 2
    for fn, packed, backward in ((fwd, 0, 0), (var, 1, 0), (bwd, 0, 1), (bvar, 1, 1)):
        assert call(fn, packed, backward, W=(1 << 22) + 1) == 2
        assert call(fn, packed, backward, n=(1 << 28) + 1, T=1) == 2

    for kw in (dict(x=None), dict(f=ODD), dict(out=p[0]), dict(out=p[1]), dict(st=None), dict(st=ODD), dict(B=0),
               dict(W=0), dict(dt=5), dict(mode=3)):
        a = dict(x=p[0], f=p[1], out=p[2], st=p[3], B=2, W=64, dt=1, mode=0)
        a.update(kw)
        assert step(a["x"], a["f"], a["out"], a["st"], a["B"], a["W"], a["dt"], a["mode"], None) == 1, kw


def test_recurrence_workspace_size(lib):
    f = lib.lightning_attn_gated_recurrence_workspace_size
    f.restype = ctypes.c_size_t
    for bad in ((0, 10, 8, 1, 0), (1, -1, 8, 1, 0), (1, 10, 0, 1, 0), (1, 10, 8, 2, 0)):
        assert f(*bad) == 0, bad
    small, back = f(2, 1000, 64, 1, 0), f(2, 1000, 64, 1, 1)
    assert small >= 256 and back >= small + 8 * 64 * 4       # the backward's own checkpoints
    assert f(1, 0, 64, 0, 0) >= 256


def _walks(lib):
    """The four calls over rows as functions of keywords, with arguments that do not meet by default."""
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    p = _ptrs(16)

    def walk(name, packed, backward):
        fn = getattr(lib, "lightning_attn_gated_recurrence" + ("_backward" if backward else "") + ("_varlen" if packed else ""))
        fn.argtypes = [vp] * ((9 if backward else 6) + packed) + [i32] * 5 + [vp, sz, vp]

        def call(**kw):
            a = dict(x=p[0], f=p[1], dout=p[2], out=p[3], df=p[4], s0=p[6], s1=p[7], ds1=p[8], ds0=p[9], ck=p[10], cu=p[5],
                     ws=WS)
            a.update(kw)
            states = ("s0", "ds1", "ds0") if backward else ("s0", "s1")
            head = ("x", "f", *(("dout", "out", "df") if backward else ("out",)), *states, "ck", *(("cu",) if packed else ()))
            return fn(*(a[k] for k in head), 2, kw.get("T", 8), 64, 1, 1, a["ws"], 1 << 40, None)
        return call
    return [(walk("", packed, backward), packed, backward) for packed in (0, 1) for backward in (0, 1)]


def test_recurrence_entries_refuse_overlaps(lib):
    """Rows are 8 * 64 bf16 values (twice that for two sequences of 8), states 2 * 64 floats; a buffer that starts inside
    another one, or ends inside it, meets it."""
    near = lambda q, by: ctypes.c_void_p(q.value + by)  # noqa: E731
    p = _ptrs(16)
    for call, packed, backward in _walks(lib):
        rows = 1024 if packed else 2048
        written = ["out", "df"] if backward else ["out"]
        others = ["x", "f"] + (["dout"] if backward else []) + written
        at = dict(x=p[0], f=p[1], dout=p[2], out=p[3], df=p[4], s0=p[6], s1=p[7], ds1=p[8], ds0=p[9], ck=p[10], cu=p[5])
        bad = [{w: near(at[o], by)} for w in written for o in others if o != w for by in (0, 16, -16, rows - 16, 16 - rows)]
        bad += [{w: near(at[o], by)} for w in written for o in ["s0", "ck"] + ["cu"] * packed for by in (0, -16)]
        bad += [dict(ck=near(at["x"], 16))] if not backward else []
        last = "ds0" if backward else "s1"
        bad += [{last: near(at[o], by)} for o in others + ["ck"] for by in (0, 16, -16)]
        bad += [dict(out=WS), {last: near(WS, 256)}]
        if backward:
            bad += [dict(ds0=near(at["s0"], by)) for by in (0, 16, -256)]
            bad += [dict(s0=at["ds1"], ds0=at["ds1"])]
        for kw in bad:
            assert call(**kw) == 1, (packed, backward, kw)
        # what may be: the final states over the initial ones, and buffers side by side (3: accepted, but there is no
        # GPU; where there is one, these addresses are not to reach it)
        if torch.cuda.is_available():
            continue
        first = at["ds1" if backward else "s0"]
        # the error record and the copy of the states: 256 bytes and 2 * 64 floats; then room for checkpoints, unused here
        for kw in ({}, {last: first}, {last: near(first, 16)}, {last: near(first, -256)}, dict(out=near(at["x"], rows)),
                   dict(out=near(at["x"], -rows)), dict(x=at["f"]), dict(ck=near(WS, 768))):
            assert call(**kw) == 3, (packed, backward, kw)


def test_recurrence_step_refuses_overlaps(lib):
    vp, i32 = ctypes.c_void_p, ctypes.c_int
    step = lib.lightning_attn_gated_recurrence_step
    step.argtypes = [vp] * 4 + [i32] * 4 + [vp]
    p = _ptrs(4)
    near = lambda q, by: vp(q.value + by)  # noqa: E731

    def call(x=p[0], f=p[1], out=p[2], state=p[3], dt=1):
        return step(x, f, out, state, 2, 64, dt, 1, None)

    for dt, row in ((0, 512), (1, 256)):
        for by in (0, 16, -16, row - 16, 16 - row):
            assert call(out=near(p[0], by), dt=dt) == 1 and call(out=near(p[1], by), dt=dt) == 1
        for by in (16, -16, row - 16, -496):
            assert call(state=near(p[0], by), dt=dt) == 1 and call(state=near(p[2], by), dt=dt) == 1
    assert call(state=p[0]) == 1 and call(state=p[2]) == 1      # bf16 values under fp32 ones
    if torch.cuda.is_available():       # accepted calls' addresses are not to reach a GPU
        return
    for kw in ({}, dict(state=p[0], dt=0), dict(state=p[2], dt=0), dict(out=near(p[0], 256)), dict(state=near(p[0], -512))):
        assert call(**kw) == 3, kw


def test_layer_norm_entries_refuse(lib):
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    fwd, bwd = lib.lightning_attn_layer_norm, lib.lightning_attn_layer_norm_backward
    fwd.argtypes = [vp] * 6 + [i32] * 3 + [f32, vp]
    bwd.argtypes = [vp] * 7 + [i32] * 3 + [f32, vp, sz, vp]
    p = _ptrs(8)

    def f(**kw):
        a = dict(x=p[0], res=None, w=None, b=None, out=p[1], sum=None, rows=4, W=64, dt=1, eps=1e-5)
        a.update(kw)
        return fwd(a["x"], a["res"], a["w"], a["b"], a["out"], a["sum"], a["rows"], a["W"], a["dt"], a["eps"], None)

    def g(**kw):
        a = dict(s=p[0], dout=p[1], dsum=None, w=None, dx=p[2], dw=p[3], db=p[4], rows=4, W=64, dt=1, eps=1e-5, ws=WS,
                 nb=1 << 30)
        a.update(kw)
        return bwd(a["s"], a["dout"], a["dsum"], a["w"], a["dx"], a["dw"], a["db"], a["rows"], a["W"], a["dt"],
                   a["eps"], a["ws"], a["nb"], None)

    for kw in (dict(x=None), dict(out=None), dict(x=ODD), dict(out=ODD), dict(res=ODD), dict(w=ODD), dict(b=ODD),
               dict(sum=ODD), dict(sum=p[1]), dict(rows=-1), dict(W=0), dict(dt=2), dict(eps=0.0),
               dict(eps=float("nan"))):
        assert f(**kw) == 1, kw
    for kw in (dict(s=None), dict(dout=None), dict(dx=None), dict(s=ODD), dict(dout=ODD), dict(dx=ODD),
               dict(dsum=ODD), dict(w=ODD), dict(dw=ODD), dict(db=ODD), dict(dw=p[4]), dict(rows=-1), dict(W=0),
               dict(dt=2), dict(eps=0.0), dict(ws=None), dict(ws=vp(0x1000010)), dict(nb=16)):
        assert g(**kw) == 1, kw
    assert f(W=16385) == 2 and g(W=16385) == 2
    assert f(rows=0, x=None, out=None) == 0                  # nothing to do
    size = lib.lightning_attn_layer_norm_workspace_size
    size.restype = ctypes.c_size_t
    assert size(-1, 64) == 0 and size(4, 0) == 0 and size(4, 16385) == 0
    assert size(0, 64) >= 256 and size(100, 64) >= 2 * 64 * 4


def test_layer_norm_entries_refuse_overlaps(lib):
    """4 rows of 64 bf16 values: 512 bytes; the weights are 256 bytes."""
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    fwd, bwd = lib.lightning_attn_layer_norm, lib.lightning_attn_layer_norm_backward
    fwd.argtypes = [vp] * 6 + [i32] * 3 + [f32, vp]
    bwd.argtypes = [vp] * 7 + [i32] * 3 + [f32, vp, sz, vp]
    p = _ptrs(8)
    near = lambda q, by: vp(q.value + by)  # noqa: E731
    at = dict(x=p[0], res=p[1], w=p[2], b=p[3], out=p[4], sum=p[5])
    grad = dict(s=p[0], dout=p[1], dsum=p[2], w=p[3], dx=p[4], dw=p[5], db=p[6], ws=WS)

    def f(**kw):
        a = {**at, **kw}
        return fwd(a["x"], a["res"], a["w"], a["b"], a["out"], a["sum"], 4, 64, 1, 1e-5, None)

    def g(**kw):
        a = {**grad, **kw}
        return bwd(a["s"], a["dout"], a["dsum"], a["w"], a["dx"], a["dw"], a["db"], 4, 64, 1, 1e-5, a["ws"], 1 << 30, None)

    off = (16, -16, 496, -496)
    bad = [{to: near(at[o], by)} for to in ("out", "sum") for o in ("x", "res") for by in off]
    bad += [{to: near(at[o], by)} for to in ("out", "sum") for o in ("w", "b") for by in (0, 16, -496, 240)]
    bad += [dict(sum=near(at["out"], by)) for by in (0, *off)]
    for kw in bad:
        assert f(**kw) == 1, kw
    bad_g = [dict(dx=near(grad[o], by)) for o in ("s", "dout", "dsum") for by in off]
    bad_g += [dict(dx=near(grad[o], by)) for o in ("w", "dw", "db", "ws") for by in (0, 16)]
    bad_g += [dict(dw=near(grad["db"], by)) for by in (0, 16, -240)] + [{k: WS} for k in ("s", "dout", "dsum", "w", "dw", "db")]
    for kw in bad_g:
        assert g(**kw) == 1, kw
    if torch.cuda.is_available():       # accepted calls' addresses are not to reach a GPU
        return
    for kw in ({}, dict(out=p[0]), dict(out=p[1]), dict(sum=p[0]), dict(out=p[0], sum=p[1]), dict(out=near(p[0], 512)),
               dict(res=p[0]), dict(b=p[2])):
        assert f(**kw) == 3, kw
    for kw in ({}, dict(dx=p[0]), dict(dx=p[1]), dict(dx=p[2]), dict(dw=p[3]), dict(dw=p[1]), dict(dx=near(p[0], -512)),
               dict(db=None)):
        assert g(**kw) == 3, kw


def test_layer_norm_workspace_is_what_the_launch_uses(lib):
    """A part of the sums, 2 W floats, for each CTA that the rows make or that fits: at most 8 on each of 148 SMs, one of
    them for wide rows."""
    if torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 148:
        pytest.skip("the numbers are for 148 SMs")
    size = lib.lightning_attn_layer_norm_workspace_size
    size.restype = ctypes.c_size_t
    up = lambda n: (n + 255) & ~255  # noqa: E731
    for rows, W, parts in ((8192, 8192, 148), (100000, 16384, 148), (256, 8192, 148), (100, 8192, 100), (100000, 512, 1184),
                           (100000, 128, 592), (64, 128, 8), (1, 16384, 1)):
        assert size(rows, W) == up(parts * 2 * W * 4), (rows, W, size(rows, W) // (8 * W))


# --------------------------------------------------------------------------- binding
def test_binding_refuses_host_tensors(lib):
    from long_context_attn_b200 import lightning_attn as la
    t = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError, match="current CUDA device"):
        la.lightning_attn_gated_recurrence(t, t, t.clone())
    with pytest.raises(ValueError, match="current CUDA device"):
        la.lightning_attn_gated_recurrence_varlen(t[0], t[0], t[0].clone(), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="current CUDA device"):
        la.lightning_attn_gated_recurrence_step(t[0], t[0], t[0].clone(), torch.zeros(4, 8))
    with pytest.raises(ValueError, match="current CUDA device"):
        la.lightning_attn_layer_norm(t, t.clone())
    with pytest.raises(ValueError, match="current CUDA device"):
        la.lightning_attn_layer_norm_backward(t, t, t.clone())


def test_binding_refuses_counts_beyond_32_bits(lib, monkeypatch):
    """2^32 + 5 rows would reach the library as 5."""
    import types

    from long_context_attn_b200 import lightning_attn as la

    class Library:
        calls, lightning_attn_status_string = [], la._lib.lightning_attn_status_string

        def __getattr__(self, name):
            return lambda *a: self.calls.append(name) or 0

    monkeypatch.setattr(la, "_check_like", lambda *a: 0)
    monkeypatch.setattr(la, "_check_cu", lambda dev, cu: cu.shape[0] - 1)
    monkeypatch.setattr(la, "_check_f32", lambda *a: None)
    st = types.SimpleNamespace(cuda_stream=0)
    t = lambda *shape: torch.empty(shape, device="meta")  # noqa: E731
    many = 2 ** 32 + 5
    calls = {
        "layer_norm": lambda n: la.lightning_attn_layer_norm(t(n, 2), t(n, 2), stream=st),
        "layer_norm_backward": lambda n: la.lightning_attn_layer_norm_backward(t(n, 2), t(n, 2), t(n, 2), stream=st),
        "gated_recurrence": lambda n: la.lightning_attn_gated_recurrence(*[t(1, n, 1)] * 3, stream=st),
        "gated_recurrence_backward": lambda n: la.lightning_attn_gated_recurrence_backward(*[t(n, 1, 1)] * 5, stream=st),
        "gated_recurrence_varlen": lambda n: la.lightning_attn_gated_recurrence_varlen(*[t(n, 1)] * 3, t(2), stream=st),
        "gated_recurrence_backward_varlen":
            lambda n: la.lightning_attn_gated_recurrence_backward_varlen(*[t(3, 1)] * 5, t(n), stream=st),
        "gated_recurrence_step": lambda n: la.lightning_attn_gated_recurrence_step(*[t(n, 1)] * 4, stream=st),
    }
    for name, call in calls.items():
        monkeypatch.setattr(la, "_lib", Library())
        call(7)
        with pytest.raises(la.LightningAttnError) as err:
            call(many)
        assert err.value.status == la.LA_ERR_UNSUPPORTED and name in str(err.value), name
    assert la._lib.calls == ["lightning_attn_" + name for name in calls]
    monkeypatch.undo()
    assert la.lightning_attn_layer_norm_workspace_size(many, 64) == 0
    assert la.lightning_attn_gated_recurrence_workspace_size(many, 10, 8, 1) == 0
    assert la.lightning_attn_gated_recurrence_workspace_size(1, many, 8, 1, True) == 0


class _Recorder:
    """Stands in for the binding: runs the fp64 references on CPU tensors."""
    from long_context_attn_b200 import lightning_attn as _la
    LA_INPUT_PLAIN, LA_INPUT_TIED = _la.LA_INPUT_PLAIN, _la.LA_INPUT_TIED

    def __init__(self):
        self.calls = []

    def _dtype(self, t):
        return 0

    def new_workspace(self, n, device=None):
        return torch.zeros(n, dtype=torch.uint8)

    def new_recurrence_checkpoints(self, tokens, W, device=None):
        return torch.zeros(-(-tokens // 128), W)

    def lightning_attn_gated_recurrence_workspace_size(self, n, tokens, W, dtype, backward=False):
        return 256

    def lightning_attn_layer_norm_workspace_size(self, rows, W):
        return 256

    def _run(self, x, f, lens, mode, s0, dout=None, ds1=None):
        n = lambda t: None if t is None else t.double().numpy()  # noqa: E731
        W = x.shape[-1]
        flat = lambda t: None if t is None else n(t).reshape(-1, W)  # noqa: E731
        return ref.packed(flat(x), flat(f), lens, mode == self.LA_INPUT_TIED, n(s0), flat(dout), n(ds1))

    def lightning_attn_gated_recurrence(self, x, f, out, s_in, s_out, saved, mode, ws):
        self.calls.append("forward" if saved is not None else "forward without checkpoints")
        r = self._run(x, f, [x.shape[1]] * x.shape[0], mode, s_in)
        out.copy_(torch.from_numpy(r["out"]).view(x.shape))
        s_out.copy_(torch.from_numpy(r["state_out"]))

    def lightning_attn_gated_recurrence_varlen(self, x, f, out, cu, s_in, s_out, saved, mode, ws):
        r = self._run(x, f, torch.diff(cu).tolist(), mode, s_in)
        out.copy_(torch.from_numpy(r["out"]))
        s_out.copy_(torch.from_numpy(r["state_out"]))

    def _grads(self, r, x, dx, df, ds_in):
        dx.copy_(torch.from_numpy(r["dx"]).view(x.shape))
        df.copy_(torch.from_numpy(r["df"]).view(x.shape))
        if ds_in is not None:
            ds_in.copy_(torch.from_numpy(r["dstate_in"]))

    def lightning_attn_gated_recurrence_backward(self, x, f, dout, dx, df, s_in, ds_out, ds_in, saved, mode, ws):
        self._grads(self._run(x, f, [x.shape[1]] * x.shape[0], mode, s_in, dout, ds_out), x, dx, df, ds_in)

    def lightning_attn_gated_recurrence_backward_varlen(self, x, f, dout, dx, df, cu, s_in, ds_out, ds_in, saved, mode,
                                                        ws):
        self._grads(self._run(x, f, torch.diff(cu).tolist(), mode, s_in, dout, ds_out), x, dx, df, ds_in)

    def lightning_attn_layer_norm(self, x, out, residual=None, sum_out=None, weight=None, bias=None, eps=1e-5):
        s = x if residual is None else x + residual
        n = lambda t: None if t is None else t.double().numpy()  # noqa: E731
        r = ref.layer_norm(n(s).reshape(-1, s.shape[-1]), n(weight), n(bias), eps)
        out.copy_(torch.from_numpy(r["out"]).view(x.shape))
        if sum_out is not None:
            sum_out.copy_(s)

    def lightning_attn_layer_norm_backward(self, s, dout, dx, dsum=None, weight=None, dweight=None, dbias=None,
                                           eps=1e-5, workspace=None):
        n = lambda t: None if t is None else t.double().numpy()  # noqa: E731
        W = s.shape[-1]
        r = ref.layer_norm(n(s).reshape(-1, W), n(weight), None, eps, n(dout).reshape(-1, W),
                           None if dsum is None else n(dsum).reshape(-1, W))
        dx.copy_(torch.from_numpy(r["dx"]).view(s.shape))
        if dweight is not None:
            dweight.copy_(torch.from_numpy(r["dweight"]))
        if dbias is not None:
            dbias.copy_(torch.from_numpy(r["dbias"]))


@pytest.fixture
def ag(monkeypatch):
    from long_context_attn_b200 import autograd
    fake = _Recorder()
    monkeypatch.setattr(autograd, "la", fake)
    autograd.fake = fake
    return autograd


def _leaf(rng, *shape):
    return torch.tensor(rng.standard_normal(shape), dtype=torch.float32, requires_grad=True)


def _plain_recurrence(x, f, lens, tied, s0):
    a = torch.sigmoid(f)
    b = (1 - a) * x if tied else x
    outs, finals, at = [], [], 0
    for i, m in enumerate(lens):
        h = torch.zeros(x.shape[1], dtype=x.dtype) if s0 is None else s0[i]
        for t in range(at, at + m):
            h = a[t] * h + b[t]
            outs.append(h)
        finals.append(h)
        at += m
    return torch.stack(outs), torch.stack(finals)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("use", ["out", "state", "both"])
def test_recurrence_autograd_wiring(ag, packed, use):
    """Gradients through either output alone or both, against torch's own autograd."""
    rng = np.random.default_rng(5)
    lens = [4, 0, 1, 6] if packed else [5, 5]
    W = 3
    x, f, s0 = _leaf(rng, sum(lens), W), _leaf(rng, sum(lens), W), _leaf(rng, len(lens), W)
    if packed:
        cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32)
        out, st = ag.gated_recurrence_varlen(x, f, cu, s0, input_mode=ag.fake.LA_INPUT_PLAIN)
    else:
        out, st = ag.gated_recurrence(x.view(2, 5, W), f.view(2, 5, W), s0, input_mode=ag.fake.LA_INPUT_PLAIN)
    wo, ws = torch.randn(sum(lens), W), torch.randn(len(lens), W)
    part = lambda o, s: {"out": (o.reshape(-1, W) * wo).sum(), "state": (s * ws).sum(),  # noqa: E731
                         "both": (o.reshape(-1, W) * wo).sum() + (s * ws).sum()}[use]
    got = torch.autograd.grad(part(out, st), (x, f, s0))
    want = torch.autograd.grad(part(*_plain_recurrence(x, f, lens, False, s0)), (x, f, s0))
    for g, w in zip(got, want):
        torch.testing.assert_close(g, w, rtol=1e-4, atol=1e-5)


def test_recurrence_without_gradients_saves_nothing(ag):
    with torch.no_grad():
        ag.gated_recurrence(torch.zeros(1, 4, 2), torch.zeros(1, 4, 2))
    assert ag.fake.calls == ["forward without checkpoints"]


@pytest.mark.parametrize("use", ["out", "sum", "both"])
def test_layer_norm_autograd_wiring(ag, use):
    rng = np.random.default_rng(6)
    x, res, w, b = _leaf(rng, 2, 3, 6), _leaf(rng, 2, 3, 6), _leaf(rng, 6), _leaf(rng, 6)
    out, s = ag.layer_norm(x, w, b, residual=res)
    wo, ws = torch.randn(2, 3, 6), torch.randn(2, 3, 6)
    part = lambda o, s: {"out": (o * wo).sum(), "sum": (s * ws).sum(), "both": (o * wo).sum() + (s * ws).sum()}[use]  # noqa: E731
    got = torch.autograd.grad(part(out, s), (x, res, w, b), allow_unused=True)
    want = torch.autograd.grad(part(torch.nn.functional.layer_norm(x + res, (6,), w, b, 1e-5), x + res),
                               (x, res, w, b), allow_unused=True)
    for g, v in zip(got, want):
        torch.testing.assert_close(g, torch.zeros_like(g) if v is None else v, rtol=1e-4, atol=1e-5)


def test_layer_norm_autograd_without_residual_or_weights(ag):
    rng = np.random.default_rng(7)
    x = _leaf(rng, 5, 6)
    y = ag.layer_norm(x)
    d = torch.randn(5, 6)
    got, = torch.autograd.grad((y * d).sum(), x)
    want, = torch.autograd.grad((torch.nn.functional.layer_norm(x, (6,)) * d).sum(), x)
    torch.testing.assert_close(got, want, rtol=1e-4, atol=1e-5)


class _StrictRecorder(_Recorder):
    """Refuses what the library refuses: tensors that are not contiguous, or not from a 16-byte boundary."""

    def __getattribute__(self, name):
        fn = super().__getattribute__(name)
        if not name.startswith("lightning_attn_") or name.endswith("_size"):
            return fn

        def call(*args, **kw):
            for t in (*args, *kw.values()):
                if torch.is_tensor(t):
                    assert t.is_contiguous() and t.data_ptr() % 16 == 0, (name, t.shape, t.data_ptr() % 16)
            return fn(*args, **kw)
        return call


@pytest.fixture
def strict(monkeypatch):
    from long_context_attn_b200 import autograd
    fake = _StrictRecorder()
    monkeypatch.setattr(autograd, "la", fake)
    autograd.fake = fake
    return autograd


@pytest.mark.parametrize("W", [7, 25, 100])
@pytest.mark.parametrize("packed", [False, True])
def test_recurrence_autograd_takes_views(strict, packed, W):
    """Slices that start off a 16-byte boundary, for every input, and such gradients (torch.cat's of parts with an odd
    number of rows): as torch's own autograd."""
    rng = np.random.default_rng(W)
    rows, lens = 5, ([2, 3] if packed else [5])
    xs, fs, ss = _leaf(rng, 1 + rows, W), _leaf(rng, 1 + rows, W), _leaf(rng, 1 + len(lens), W)
    wo, ws = torch.randn(3 + rows, W), torch.randn(1 + len(lens), W)

    def loss(run):
        x, f, s = xs[1:], fs[1:], ss[1:]
        out, st = run(x, f, s)
        return (torch.cat((torch.tanh(xs[:3]), out)) * wo).sum() + (torch.cat((ss[:1], st)) * ws).sum()

    def ours(x, f, s):
        if packed:
            cu = torch.tensor([-1, 0, 2, 5], dtype=torch.int32)[1:]
            return strict.gated_recurrence_varlen(x, f, cu, s, input_mode=strict.fake.LA_INPUT_PLAIN)
        out, st = strict.gated_recurrence(x[None], f[None], s, input_mode=strict.fake.LA_INPUT_PLAIN)
        return out[0], st

    got = torch.autograd.grad(loss(ours), (xs, fs, ss))
    want = torch.autograd.grad(loss(lambda x, f, s: _plain_recurrence(x, f, lens, False, s)), (xs, fs, ss))
    for g, w in zip(got, want):
        torch.testing.assert_close(g, w, rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("W", [7, 25, 100])
def test_layer_norm_autograd_takes_views(strict, W):
    rng = np.random.default_rng(W)
    xs, rs, wb = _leaf(rng, 6, W), _leaf(rng, 6, W), _leaf(rng, 1 + 2 * W)
    wo, ws = torch.randn(8, W), torch.randn(8, W)

    def loss(run):
        out, s = run(xs[1:], wb[1:1 + W], wb[1 + W:], rs[1:])
        return (torch.cat((xs[:3], out)) * wo).sum() + (torch.cat((rs[:3], s)) * ws).sum()

    got = torch.autograd.grad(loss(lambda x, w, b, r: strict.layer_norm(x, w, b, residual=r)), (xs, rs, wb))
    want = torch.autograd.grad(loss(lambda x, w, b, r: (torch.nn.functional.layer_norm(x + r, (W,), w, b, 1e-5), x + r)),
                               (xs, rs, wb))
    for g, w in zip(got, want):
        torch.testing.assert_close(g, w, rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("packed", [False, True])
def test_recurrence_autograd_uses_the_callers_workspace(ag, packed, monkeypatch):
    """The error record of the forward and of the backward is where the caller can read it."""
    seen = []

    def note(name):
        real = getattr(ag.fake, name)
        monkeypatch.setattr(ag.fake, name, lambda *a: (seen.append(a[-1]), real(*a))[1])

    tail = "_varlen" if packed else ""
    note("lightning_attn_gated_recurrence" + tail)
    note("lightning_attn_gated_recurrence_backward" + tail)
    x, ws = torch.zeros(1, 4, 2, requires_grad=True), torch.zeros(4096, dtype=torch.uint8)
    for given in (ws, None):
        if packed:
            out, _ = ag.gated_recurrence_varlen(x[0], x[0], torch.tensor([0, 4], dtype=torch.int32), workspace=given)
        else:
            out, _ = ag.gated_recurrence(x, x, workspace=given)
        out.sum().backward()
    assert len(seen) == 4 and all(w is ws for w in seen[:2]) and all(w is not ws and w is not None for w in seen[2:])
