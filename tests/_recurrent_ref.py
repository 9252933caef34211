"""The gated recurrence and the layer norm in fp64 (numpy, straight from the formulas), with
bounds on the error that fp32 arithmetic and one rounding to the output type can make.

Every bound is a first-order sum over the roundings of the computation, u = 2^-24 being the
relative error of one fp32 operation:

  gate   t = exp(-f) is off by at most 4u with expf (2 ulp, the bound CUDA states), and by (4 + |f|)u
         where exp2 is taken of the rounded product -f log2(e) (bf16 gates). 1 + t adds u, the
         reciprocal after its Newton step 2u, a product u. t's error reaches a = 1 / (1 + t) times
         t / (1 + t): for f >= 0 that is at most 2u + 0.28u (|f| t / (1 + t) <= 0.28), so a is
         within 6u there, and a for f < 0 and 1 - a within (8 + |f|)u.
  scan   h_t is a sum of terms (a_{s+1} .. a_t) b_s.  A term takes at most t - s + 1 gates and as many
         products, whatever their order (a tree over tiles multiplies the same factors): 16u for
         each covers 6u + u, and gates down to f = -9. What gates below that add, |f| - 9 each, sums
         to less than 88u as long as the term is a normal fp32 number (its size is at most the product
         of their exp(-|f|) > 2^-126 = exp(-87.3)). With M_t = a_t M_{t-1} + |b_t| and
         N_t = a_t N_{t-1} + M_t (so that N_t = sum over s of (t - s + 1) times the term's size) all of
         it is inside 16u N_t + 88u M_t. Adding the terms up rounds each partial sum once per level:
         at most 16 rows of a thread, 3 of a warp's groups, 8 warps and 16 tiles of a round, 43 levels;
         88u + 43u < 200u M_t.  Further tiles add a level for each 128 rows or more, inside the spare
         of 16u for each row.
  out    one rounding to the output type: half an eps of the value.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def sigmoid(f):
    e = np.exp(-np.abs(f))
    return np.where(f >= 0, 1 / (1 + e), e / (1 + e))


def scan(a, b, h):
    """h_t = a_t h_{t-1} + b_t over the first axis: all h_t."""
    out = np.empty_like(b)
    for t in range(b.shape[0]):
        h = a[t] * h + b[t]
        out[t] = h
    return out


def scan_bound(a, b, h0):
    """Bound on the fp32 error of scan()'s h_t (before any rounding), with M_t."""
    M = scan(a, np.abs(b), np.abs(h0))
    N = scan(a, M, np.abs(h0))
    return U * (16 * N + 200 * M), M


def sequence(x, f, tied, s0=None, dout=None, ds1=None):
    """One sequence x, f [T, W] (fp64): dict of the forward's and, with dout, the backward's
    values, and under the same names + "_tol" what fp32 arithmetic may be off by."""
    T, W = x.shape
    s0 = np.zeros(W) if s0 is None else s0
    a, keep = sigmoid(f), sigmoid(-f)
    b = keep * x if tied else x
    h = scan(a, b, s0)
    tol, M = scan_bound(a, b, s0)
    r = dict(out=h, out_tol=tol, state_out=h[-1] if T else s0, state_out_tol=tol[-1] if T else np.zeros(W))
    prev = np.concatenate((s0[None], h))[:T]
    prev_tol = np.concatenate((np.zeros((1, W)), tol))[:T]
    prev_M = np.concatenate((np.abs(s0)[None], M))[:T]
    r["enter"], r["enter_tol"] = prev, prev_tol
    if dout is None:
        return r
    ds1 = np.zeros(W) if ds1 is None else ds1
    # c_t = a_t (dout_t + c_{t+1}), G_t = dout_t + c_{t+1}
    ar, dr = a[::-1], dout[::-1]
    c = scan(ar, ar * dr, ds1)[::-1]
    ctol, cM = (t[::-1] for t in scan_bound(ar, ar * dr, ds1))
    nxt = np.concatenate((c, ds1[None]))[1:]
    G = dout + nxt
    Gtol = np.concatenate((ctol, np.zeros((1, W))))[1:] + U * np.abs(G)
    Gabs = np.abs(dout) + np.concatenate((cM, np.abs(ds1)[None]))[1:]
    d = prev - x if tied else prev
    dabs = prev_M + np.abs(x) if tied else prev_M
    slope = a * keep
    r["dx"] = keep * G if tied else G
    r["dx_tol"] = (keep if tied else 1.0) * (Gtol + 10 * U * Gabs)
    r["df"] = slope * G * d
    r["df_tol"] = slope * (Gtol * dabs + Gabs * (prev_tol + U * dabs) + 24 * U * Gabs * dabs)
    r["dstate_in"] = c[0] if T else ds1
    r["dstate_in_tol"] = ctol[0] if T else np.zeros(W)
    return r


def packed(x, f, lens, tied, s0=None, dout=None, ds1=None):
    """Sequences of `lens` rows one after the other in x, f [rows, W]: per-token values packed,
    states stacked."""
    parts, at = [], 0
    for i, m in enumerate(lens):
        cut = slice(at, at + m)
        parts.append(sequence(x[cut], f[cut], tied, None if s0 is None else s0[i],
                              None if dout is None else dout[cut], None if ds1 is None else ds1[i]))
        at += m
    join = lambda k, v: np.stack(v) if "state" in k else np.concatenate(v)  # noqa: E731
    return {k: join(k, [p[k] for p in parts]) for k in parts[0]}


def layer_norm(s, w, b, eps, dout=None, dsum=None):
    """Rows s [rows, W] (fp64): dict of out and, with dout, dx, dweight, dbias, each with its
    bound.  A sum of W values rounds partial sums at most 32 times in a thread (16 vectors of one
    value, or 4 of 8 in pairs), 5 in a warp and 5 over the warps: 128u of the sum of sizes covers
    it. sqrt and the divisions are IEEE-rounded: r is within 8u more than half the variance's."""
    rows, W = s.shape
    k = 128 * U
    mean = s.mean(1, keepdims=True)
    mabs = np.abs(s).mean(1, keepdims=True)
    dev = s - mean
    dev_tol = k * mabs + U * (np.abs(s) + np.abs(dev))
    var = (dev * dev).mean(1, keepdims=True)
    r = 1 / np.sqrt(var + eps)
    # relative error of r: half that of var + eps
    r_rel = 0.5 * ((2 * np.abs(dev) * dev_tol).mean(1, keepdims=True) + k * var) * r * r + 8 * U
    z = dev * r
    z_tol = dev_tol * r + np.abs(z) * (r_rel + 2 * U)
    w = np.ones(W) if w is None else w
    b = np.zeros(W) if b is None else b
    q = dict(out=z * w + b, out_tol=z_tol * np.abs(w) + 2 * U * (np.abs(z * w) + np.abs(b)))
    if dout is None:
        return q
    g = dout * w
    mg, gabs = g.mean(1, keepdims=True), np.abs(g).mean(1, keepdims=True)
    mgz, gzabs = (g * z).mean(1, keepdims=True), np.abs(g * z).mean(1, keepdims=True)
    mgz_tol = (np.abs(g) * z_tol).mean(1, keepdims=True) + k * gzabs
    inner = g - mg - z * mgz
    inner_tol = k * gabs + np.abs(z) * mgz_tol + z_tol * np.abs(mgz) + 4 * U * (np.abs(g) + np.abs(mg) + np.abs(z * mgz))
    dx = r * inner + (0 if dsum is None else dsum)
    q["dx"] = dx
    q["dx_tol"] = r * inner_tol + np.abs(r * inner) * (r_rel + 2 * U) + U * np.abs(dx)
    # the sum over the rows: at most rows + 16 roundings of partial sums
    n = (rows + 16) * U
    q["dweight"], q["dbias"] = (dout * z).sum(0), dout.sum(0)
    q["dweight_tol"] = (np.abs(dout) * z_tol).sum(0) + n * np.abs(dout * z).sum(0)
    q["dbias_tol"] = n * np.abs(dout).sum(0)
    return q


def check(name, got, want, tol, dtype="f32"):
    """|got - want| <= tol + half a step of `dtype`, element by element."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    allowed = tol + HALF[dtype] * (np.abs(want) + tol) + 1e-37   # results below fp32's normal range
    bad = ~(np.abs(got - want) <= allowed)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) / allowed, 0)), want.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} off; at {i}: got {got[i]!r}, want {want[i]!r}, "
                             f"allowed {np.broadcast_to(allowed, want.shape)[i]:.3e}")
