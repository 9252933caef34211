"""Cases of the gated linear recurrence and the layer norm, for timing and for comparing outputs.

The gated linear recurrence (channel by channel; x, f and h have W channels a token):

    a_t = sigmoid(f_t),   b_t = x_t ("plain") or (1 - a_t) x_t ("tied"),   h_t = a_t h_{t-1} + b_t

and its backward pass, with G_t the gradient reaching h_t (after the last token: the final state's gradient):

    G_t = dout_t + a_{t+1} G_{t+1},   dx = G or (1 - a) G,   df = G a (1 - a) (h_{t-1} or h_{t-1} - x_t)

The layer norm, over the W values of a row s = x + residual:

    y = (s - mean) / sqrt(var + eps) * w + b

and its backward pass. `own` chooses between the plain form (elementary torch operations in 32 bits) and the calls
of long_context_attn_b200.
"""
import math
import random

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # The long prompt of the library's benchmark (131072 tokens of 64 heads of 128), final state kept for decoding.
        dict(name="rec_128k", op="rec", batch=1, tokens=131072, width=8192, dtype="bf16", tied=True, state=False),
        # The same prompt continued from a state, on one rank's 8 heads: few channels, so the time axis has to be split.
        dict(name="rec_128k_narrow", op="rec", batch=1, tokens=131072, width=1024, dtype="bf16", tied=True, state=True),
        # A packed batch of 16 prompts of 1000 to 32768 tokens (the benchmark's), 8 heads of 128.
        dict(name="rec_varlen16", op="rec_varlen", seqs=16, shortest=1000, longest=32768, lens_seed=16, width=1024,
             dtype="bf16", tied=False, state=True),
        # The smallest call: 512 tokens of 2 heads of 64 in fp32, where the launches are what counts.
        dict(name="rec_tiny_f32", op="rec", batch=1, tokens=512, width=128, dtype="f32", tied=False, state=False),
        # One new token for each of 256 sequences, 64 heads of 128: the decode step.
        dict(name="rec_step_256", op="rec_step", batch=256, width=8192, dtype="bf16", tied=True),
        # A training step of one 8192-token sequence, 64 heads of 128: forward, then backward.
        dict(name="rec_train_8k", op="rec_train", batch=1, tokens=8192, width=8192, dtype="bf16", tied=True,
             state=False),
        # Training on ragged, short packed sequences, 12 heads of 64 in fp32, with state gradients (truncated
        # back-propagation through time).
        dict(name="rec_train_varlen_f32", op="rec_train_varlen", seqs=101, shortest=0, longest=1200, lens_seed=7,
             width=768, dtype="f32", tied=False, state=True),
        # The pre-norm of 8192 tokens with the residual sum kept.
        dict(name="ln_8k", op="ln", rows=8192, width=8192, dtype="bf16", residual=True),
        # The pre-norm of one decode step: 256 tokens.
        dict(name="ln_step_256", op="ln", rows=256, width=8192, dtype="bf16", residual=True),
        # A single token.
        dict(name="ln_one", op="ln", rows=1, width=8192, dtype="bf16", residual=False),
        # The backward of the 8192-token pre-norm, the gradient of the residual sum added on the way.
        dict(name="ln_bwd_8k", op="ln_bwd", rows=8192, width=8192, dtype="bf16", residual=True),
        # Narrow rows in fp32, an odd number of them.
        dict(name="ln_bwd_narrow_f32", op="ln_bwd", rows=65537, width=768, dtype="f32", residual=False),
    ]


def _log_uniform(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(["rec", "rec", "rec_varlen", "rec_step", "rec_train", "rec_train_varlen", "ln", "ln", "ln_bwd",
                     "ln_bwd"])
    width = 8 * _log_uniform(rng, 16, 1024)
    case = dict(op=op, width=width, dtype=rng.choice(["bf16", "bf16", "f32"]))
    most = (1 << 27) // width                       # rows: a drawn case has at most 2^27 values a tensor
    if op.startswith("ln"):
        case.update(rows=_log_uniform(rng, 1, min(most, 300000)), residual=rng.random() < 0.5)
    elif op == "rec_step":
        case.update(batch=_log_uniform(rng, 1, min(most, 1024)), tied=rng.random() < 0.5)
    elif op.endswith("varlen"):
        seqs = _log_uniform(rng, 1, 200)
        longest = _log_uniform(rng, 8, min(32768, max(8, most // seqs)))
        case.update(seqs=seqs, shortest=rng.choice([0, 1, longest // 3]), longest=longest,
                    lens_seed=rng.randrange(1 << 20), tied=rng.random() < 0.5, state=rng.random() < 0.5)
    else:
        batch = _log_uniform(rng, 1, 64)
        case.update(batch=batch, tokens=_log_uniform(rng, 2, min(131072, most // batch)), tied=rng.random() < 0.5,
                    state=rng.random() < 0.5)
    return case


def lengths(case):
    """The sequences' lengths of a case of the recurrence."""
    if "seqs" in case:
        rng = random.Random(case["lens_seed"])
        lens = [rng.randint(case["shortest"], case["longest"]) for _ in range(case["seqs"])]
        return lens if sum(lens) else lens[:-1] + [case["longest"]]
    return [case.get("tokens", 1)] * case["batch"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, W = TYPES[case["dtype"]], case["width"]

    def normal(*shape, scale=1.0, dtype=dt):
        t = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)
        return t if scale == 1.0 else t.mul_(scale)

    st = dict(case=case)
    if case["op"].startswith("ln"):
        rows = case["rows"]
        # Rows as a residual stream has them: a mean and a scale of their own.
        st["x"] = normal(rows, W).mul_(normal(rows, 1).abs_().add_(0.5)).add_(normal(rows, 1))
        st["w"] = normal(W, scale=0.2, dtype=torch.float32).add_(1.0)
        st["out"] = torch.empty_like(st["x"])
        if case["op"] == "ln":
            st["b"] = normal(W, scale=0.1, dtype=torch.float32)
            if case["residual"]:
                st["res"] = normal(rows, W, scale=0.5)
                st["sum"] = torch.empty_like(st["x"])
        else:
            st["dout"] = normal(rows, W)
            st["dsum"] = normal(rows, W) if case["residual"] else None
            st["dw"] = torch.empty(W, dtype=torch.float32, device="cuda")
            st["db"] = torch.empty(W, dtype=torch.float32, device="cuda")
        return st
    lens = lengths(case)
    n, rows = len(lens), sum(lens)
    packed = "seqs" in case
    shape = (rows, W) if packed or case["op"] == "rec_step" else (n, case["tokens"], W)
    st["x"] = normal(*shape)
    # Forget gates with a bias of each channel's own, so that channels remember from 2 to about 1000 tokens.
    st["f"] = normal(*shape).add_(torch.empty(W, dtype=dt, device="cuda").uniform_(0.0, 7.0, generator=gen))
    st["out"] = torch.empty_like(st["x"])
    if packed:
        cu = [0]
        for m in lens:
            cu.append(cu[-1] + m)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["op"] == "rec_step":
        st["state"] = normal(n, W, dtype=torch.float32)
        return st
    st["s0"] = normal(n, W, dtype=torch.float32) if case["state"] else None
    st["s1"] = torch.empty(n, W, dtype=torch.float32, device="cuda")
    if "train" in case["op"]:
        st["dout"] = normal(*shape)
        st["dx"], st["df"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        if case["state"]:
            st["ds1"] = normal(n, W, dtype=torch.float32)
            st["ds0"] = torch.empty(n, W, dtype=torch.float32, device="cuda")
    return st


# ---------------------------------------------------------------------------------------
# Plain form
# ---------------------------------------------------------------------------------------
def _scan(a, b, longest):
    """h[t] = a[t] h[t-1] + b[t] along the rows (a is 0 where a sequence starts), by doubling the reach."""
    reach = 1
    while reach < longest:
        b = torch.cat((b[:reach], torch.addcmul(b[reach:], a[reach:], b[:-reach])))
        a = torch.cat((a[:reach], a[reach:] * a[:-reach]))
        reach *= 2
    return b


def _bounds(st):
    """First and last row of each sequence that has any, and which sequences these are."""
    if "cu" in st:
        cu = st["cu"].long()
        some = (cu[1:] > cu[:-1]).nonzero()[:, 0]
        return cu[:-1][some], cu[1:][some] - 1, some
    n, T = st["x"].shape[:2]
    some = torch.arange(n, device="cuda")
    return some * T, some * T + T - 1, some


def _forward(st, longest):
    """sigmoid(f), h and the final states, in 32 bits, over packed rows."""
    W = st["x"].shape[-1]
    x, f = st["x"].reshape(-1, W).float(), st["f"].reshape(-1, W).float()
    a = torch.sigmoid(f)
    b = torch.sigmoid(-f).mul_(x) if st["case"]["tied"] else x.clone()
    first, last, some = _bounds(st)
    s0 = st["s0"]
    if s0 is not None:
        b[first] += a[first] * s0[some]
    decay = a.clone()
    decay[first] = 0.0
    h = _scan(decay, b, longest)
    final = torch.zeros_like(st["s1"]) if s0 is None else s0.clone()
    final[some] = h[last]
    return x, f, a, h, final


def _train(st, longest):
    x, f, a, h, final = _forward(st, longest)
    first, last, some = _bounds(st)
    W = x.shape[1]
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    prev[first] = 0.0 if st["s0"] is None else st["s0"][some]
    grad = st["dout"].reshape(-1, W).float().clone()
    if st.get("ds1") is not None:
        grad[last] += st["ds1"][some]
    decay = torch.zeros_like(a)
    decay[:-1] = a[1:]
    decay[last] = 0.0
    grad = _scan(decay.flip(0), grad.flip(0), longest).flip(0)
    keep = torch.sigmoid(-f)
    if st["case"]["tied"]:
        dx, df = grad * keep, grad * a * keep * (prev - x)
    else:
        dx, df = grad, grad * a * keep * prev
    got = [h, final, dx, df]
    if st.get("ds1") is not None:
        ds0 = st["ds1"].clone()
        ds0[some] = a[first] * grad[first]
        got.append(ds0)
    return got


def _plain(st):
    case = st["case"]
    op, shape, dt = case["op"], st["x"].shape, st["x"].dtype
    if op == "rec_step":
        f = st["f"].float()
        b = st["x"].float() if not case["tied"] else torch.sigmoid(-f) * st["x"].float()
        st["state"].mul_(torch.sigmoid(f)).add_(b)
        return [st["state"].to(dt), st["state"]]
    if op.startswith("rec_train"):
        got = _train(st, max(lengths(case)))
        return [got[0].to(dt).reshape(shape), got[1], got[2].to(dt).reshape(shape), got[3].to(dt).reshape(shape)] + got[4:]
    if op.startswith("rec"):
        h, final = _forward(st, max(lengths(case)))[3:]
        return [h.to(dt).reshape(shape), final]
    s = st["x"].float()
    if "res" in st:
        s = s + st["res"].float()
    mean = s.mean(-1, keepdim=True)
    xhat = s - mean
    r = torch.rsqrt((xhat * xhat).mean(-1, keepdim=True) + EPS)
    xhat = xhat * r
    if op == "ln":
        y = (xhat * st["w"] + st["b"]).to(dt)
        return [y, s.to(dt)] if "res" in st else [y]
    dy = st["dout"].float()
    g = dy * st["w"]
    dx = r * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    return [dx.to(dt), (dy * xhat).sum(0), dy.sum(0)]


# ---------------------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------------------
def _own(st):
    from long_context_attn_b200 import lightning_attn as la
    case = st["case"]
    op = case["op"]
    if op == "ln":
        la.lightning_attn_layer_norm(st["x"], st["out"], residual=st.get("res"), sum_out=st.get("sum"),
                                     weight=st["w"], bias=st["b"], eps=EPS)
        return [st["out"], st["sum"]] if "res" in st else [st["out"]]
    if op == "ln_bwd":
        if "ws" not in st:      # kept for the passes that follow, as a program keeps it
            st["ws"] = la.new_workspace(la.lightning_attn_layer_norm_workspace_size(case["rows"], case["width"]))
        la.lightning_attn_layer_norm_backward(st["x"], st["dout"], st["out"], dsum=st["dsum"], weight=st["w"],
                                              dweight=st["dw"], dbias=st["db"], eps=EPS, workspace=st["ws"])
        return [st["out"], st["dw"], st["db"]]
    mode = la.LA_INPUT_TIED if case["tied"] else la.LA_INPUT_PLAIN
    if op == "rec_step":
        la.lightning_attn_gated_recurrence_step(st["x"], st["f"], st["out"], st["state"], input_mode=mode)
        return [st["out"], st["state"]]
    train = "train" in op
    if "ws" not in st:          # kept for the passes that follow, as a program keeps it
        W = case["width"]
        rows = st["x"].numel() // W
        st["ws"] = la.new_workspace(la.lightning_attn_gated_recurrence_workspace_size(
            st["s1"].shape[0], rows, W, la._dtype(st["x"]), train))
        st["saved"] = la.new_recurrence_checkpoints(rows, W) if train else None
    kw = dict(state_in=st["s0"], input_mode=mode, checkpoints=st["saved"], workspace=st["ws"])
    if "cu" in st:
        la.lightning_attn_gated_recurrence_varlen(st["x"], st["f"], st["out"], st["cu"], state_out=st["s1"], **kw)
    else:
        la.lightning_attn_gated_recurrence(st["x"], st["f"], st["out"], state_out=st["s1"], **kw)
    got = [st["out"], st["s1"]]
    if train:
        kw.update(dstate_out=st.get("ds1"), dstate_in=st.get("ds0"))
        if "cu" in st:
            la.lightning_attn_gated_recurrence_backward_varlen(st["x"], st["f"], st["dout"], st["dx"], st["df"],
                                                               st["cu"], **kw)
        else:
            la.lightning_attn_gated_recurrence_backward(st["x"], st["f"], st["dout"], st["dx"], st["df"], **kw)
        got += [st["dx"], st["df"]] + ([st["ds0"]] if "ds0" in st else [])
    return got


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    W, e = case["width"], SIZE[case["dtype"]]
    if case["op"].startswith("ln"):
        n = case["rows"] * W
        if case["op"] == "ln":      # x (and the residual) in, y (and the sum) out
            return dict(bytes=n * e * (4 if case["residual"] else 2) + 8 * W, flops=8 * n)
        return dict(bytes=n * e * (4 if case["residual"] else 3) + 12 * W, flops=16 * n)
    lens = lengths(case)
    n, states = sum(lens) * W, len(lens) * W * 4
    if case["op"] == "rec_step":
        return dict(bytes=3 * n * e + 2 * states, flops=8 * n)
    # x, f in, h and the final states out; a training step: dout in, dx and df out, and the states' gradients
    both = 1 + case["state"]
    if "train" in case["op"]:
        return dict(bytes=6 * n * e + (both + 2 * case["state"]) * states, flops=24 * n)
    return dict(bytes=3 * n * e + both * states, flops=8 * n)


# ---------------------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------------------
def _exact_recurrence(a, b, h):
    """h[t] = a[t] h[t-1] + b[t] token by token over the first axis, from h."""
    out = torch.empty_like(b)
    for t in range(b.shape[0]):
        h = torch.addcmul(b[t], a[t], h, out=out[t])
    return out


def _exact_layer(x, f, tied, s0, dout=None, ds1=None):
    """One batch of equally long sequences, time first: h, the final state, and the gradients where dout is given."""
    e = torch.exp(-f)
    a = 1 / (1 + e)
    keep = e / (1 + e)
    h = _exact_recurrence(a, keep * x if tied else x, s0)
    if dout is None:
        return h, h[-1]
    prev = torch.cat((s0[None], h[:-1]))
    # c_t = a_t (dout_t + c_{t+1}): what flows from token t back to the state before it
    c = _exact_recurrence(a.flip(0), (a * dout).flip(0), ds1).flip(0)
    G = dout + torch.cat((c[1:], ds1[None]))
    slope = a * keep * G
    return h, h[-1], keep * G if tied else G, slope * (prev - x) if tied else slope * prev, c[0]


def exact(case, seed):
    st = prepare(case, seed)
    W = case["width"]
    if case["op"].startswith("ln"):
        s = st["x"].double()
        if "res" in st:
            s += st["res"]
        var, mean = torch.var_mean(s, dim=-1, correction=0, keepdim=True)
        std = (var + EPS).sqrt()
        z = (s - mean) / std
        if case["op"] == "ln":
            y = torch.addcmul(st["b"].double(), z, st["w"].double())
            return [y, s] if "res" in st else [y]
        dy = st["dout"].double()
        dz = dy * st["w"].double()
        dx = (dz - dz.mean(-1, keepdim=True) - z * torch.einsum("rc,rc->r", dz, z)[:, None] / W) / std
        if st["dsum"] is not None:
            dx += st["dsum"]
        return [dx, torch.einsum("rc,rc->c", dy, z), dy.sum(0)]
    if case["op"] == "rec_step":
        h = _exact_layer(st["x"].double()[None], st["f"].double()[None], case["tied"], st["state"].double())[1]
        return [h, h]
    lens = lengths(case)
    steps = sum(lens) if "seqs" in case else case["tokens"]
    if steps * (3 if "train" in case["op"] else 1) > 800000:     # the loop over tokens would take too long
        return None
    train, n = "train" in case["op"], len(lens)
    zero = torch.zeros(n, W, dtype=torch.float64, device="cuda")
    s0 = zero if st["s0"] is None else st["s0"].double()
    ds1 = st["ds1"].double() if st.get("ds1") is not None else zero
    if "seqs" not in case:
        first = lambda k: st[k].double().transpose(0, 1).contiguous() if train or k != "dout" else None  # noqa: E731
        got = _exact_layer(first("x"), first("f"), case["tied"], s0, first("dout"), ds1)
        got = [t.transpose(0, 1) if i != 1 and i != 4 else t for i, t in enumerate(got)]
    else:
        parts, at = [], 0
        for i, m in enumerate(lens):
            cut = lambda k: st[k][at:at + m].double()  # noqa: E731
            if m:
                parts.append(_exact_layer(cut("x"), cut("f"), case["tied"], s0[i], cut("dout") if train else None, ds1[i]))
            else:
                none = st["x"][:0].double()
                parts.append((none, s0[i], none, none, ds1[i])[:5 if train else 2])
            at += m
        got = [torch.stack(p) if i in (1, 4) else torch.cat(p) for i, p in enumerate(zip(*parts))]
    return list(got) if "ds0" in st else list(got)[:4]
