"""fp64 oracle of the selective state space scan, its short causal convolution
and the norms around a block, with their gradients.

TEST INFRASTRUCTURE ONLY: nothing in the library's compute path may import or
call this module; only the test suite and the smoke check do.  It shares no
code with the CUDA path.

Each function takes fp32 values (widened) and works token by token.  With
``mag=True`` it returns magnitudes instead of values: every product and sum
over absolute values, with the decays as they are.  A result computed in
floating point is off by at most (roundings on its longest path) x 2^-24 x its
magnitude, which is what the tests hold the kernels to.
"""
from __future__ import annotations

import numpy as np


def _f(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def softplus(v):
    with np.errstate(invalid="ignore"):  # NaN stays NaN
        return np.logaddexp(0.0, v)


def sigmoid(v):
    return np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))


def silu(v):
    return v * sigmoid(v)


def dsilu(v):
    s = sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


def dsilu_mag(v):
    """Magnitude of silu's slope.  Its two terms cancel near v = -1.28: the
    computed sum is off by roundings of s and of s v (1 - s), which stay of
    size 0.2 there while the slope itself goes through zero, so |dsilu(v)|
    would bound nothing."""
    s = sigmoid(v)
    return s * (1.0 + np.abs(v) * (1.0 - s))


def _channels(m, E):
    """[..., G, N] of the groups as [..., E, N] of the channels."""
    return np.repeat(m, E // m.shape[-2], axis=-2)


def _groups(m, G):
    """Sums over each group's channels: [..., E, N] -> [..., G, N]."""
    s = m.shape
    return m.reshape(s[:-2] + (G, s[-2] // G, s[-1])).sum(-2)


def scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus_dt=True, h0=None, lens=None,
         out=None, mag=False):
    """y [B, L, E] and the state after the last token [B, E, N].  Rows behind
    lens[b] keep the values of ``out`` (zeros without it)."""
    x, dt, A, Bm, Cm, D, z, dt_bias, h0 = map(_f, (x, dt, A, Bm, Cm, D, z, dt_bias, h0))
    m = np.abs if mag else (lambda v: v)
    B, L, E = x.shape
    step = dt if dt_bias is None else dt + dt_bias
    step = softplus(step) if softplus_dt else step
    h = np.zeros((B, E, A.shape[1])) if h0 is None else m(h0).copy()
    y = np.zeros((B, L, E)) if out is None else _f(out).copy()
    for b in range(B):
        for t in range(L if lens is None else int(np.clip(lens[b], 0, L))):
            u = m(step[b, t] * x[b, t])
            h[b] = np.exp(step[b, t][:, None] * A) * h[b] + u[:, None] * m(_channels(Bm[b, t], E))
            v = (h[b] * m(_channels(Cm[b, t], E))).sum(-1)
            if D is not None:
                v = v + m(D * x[b, t])
            y[b, t] = v if z is None else v * m(silu(z[b, t]))
    return y, h


def scan_step(x, dt, A, Bm, Cm, h, D=None, z=None, dt_bias=None, softplus_dt=True, mag=False):
    """One token: y [B, E] and the state behind it."""
    one = lambda v: None if v is None else np.asarray(v)[:, None]  # noqa: E731
    y, h = scan(one(x), one(dt), A, one(Bm), one(Cm), D, one(z), dt_bias, softplus_dt, h, mag=mag)
    return y[:, 0], h


def scan_backward(x, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, softplus_dt=True, h0=None,
                  dh=None, mag=False):
    """dict of the gradients dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0."""
    x, dt, A, Bm, Cm, dy, D, z, dt_bias, h0, dh = map(
        _f, (x, dt, A, Bm, Cm, dy, D, z, dt_bias, h0, dh))
    m = np.abs if mag else (lambda v: v)
    B, L, E = x.shape
    G, N = Bm.shape[-2:]
    raw = dt if dt_bias is None else dt + dt_bias
    step = softplus(raw) if softplus_dt else raw
    hs = np.zeros((B, L + 1, E, N))
    if h0 is not None:
        hs[:, 0] = m(h0)
    decay = np.exp(step[..., None] * A)
    u = m(step * x)
    Be, Ce = m(_channels(Bm, E)), m(_channels(Cm, E))
    for t in range(L):
        hs[:, t + 1] = decay[:, t] * hs[:, t] + u[:, t, :, None] * Be[:, t]
    gy = m(dy) if z is None else m(dy * silu(z))
    got = {k: np.zeros_like(x) for k in ("dx", "ddt")}
    got["dA"] = np.zeros_like(A)
    got["dB"], got["dC"] = np.zeros(Bm.shape), np.zeros(Cm.shape)
    after = np.zeros((B, E, N)) if dh is None else m(dh)  # dL/dh_t from later tokens
    for t in range(L - 1, -1, -1):
        g = Ce[:, t] * gy[:, t, :, None] + after
        got["dC"][:, t] = _groups(hs[:, t + 1] * gy[:, t, :, None], G)
        got["dB"][:, t] = _groups(g * u[:, t, :, None], G)
        du = (g * Be[:, t]).sum(-1)
        w = g * decay[:, t] * hs[:, t]
        got["dx"][:, t] = du * m(step[:, t]) + (0 if D is None else m(D) * gy[:, t])
        got["ddt"][:, t] = (w * m(A)).sum(-1) + du * m(x[:, t])
        got["dA"] += (w * m(step[:, t])[..., None]).sum(0)
        after = g * decay[:, t]
    if softplus_dt:
        got["ddt"] *= sigmoid(raw)
    y = (hs[:, 1:] * Ce).sum(-1) + (0 if D is None else m(D * x))
    got["dD"] = None if D is None else (gy * m(x)).sum((0, 1))
    got["dz"] = None if z is None else m(dy) * y * (dsilu_mag(z) if mag else dsilu(z))
    got["ddt_bias"] = None if dt_bias is None else got["ddt"].sum((0, 1))
    got["dh0"] = None if h0 is None else after
    return got


def _taps(x, state, W):
    """Rows with the state's W - 1 in front: [B, W - 1 + L, E]."""
    B, _, E = x.shape
    return np.concatenate([np.zeros((B, W - 1, E)) if state is None else state, x], 1)


def conv(x, w, bias=None, silu_act=True, state=None, lens=None, out=None, mag=False):
    """y [B, L, E] and the last W - 1 rows."""
    x, w, bias, state = map(_f, (x, w, bias, state))
    m = np.abs if mag else (lambda v: v)
    B, L, E = x.shape
    W = w.shape[1]
    rows = _taps(x, state, W)
    y = np.zeros((B, L, E)) if out is None else _f(out).copy()
    last = np.zeros((B, W - 1, E))
    for b in range(B):
        n = L if lens is None else int(np.clip(lens[b], 0, L))
        for t in range(n):
            terms = rows[b, t:t + W] * w.T
            pre = terms.sum(0) + (0 if bias is None else bias)
            if mag:  # silu's slope is at most 1.1
                y[b, t] = np.abs(terms).sum(0) + (0 if bias is None else np.abs(bias))
            else:
                y[b, t] = silu(pre) if silu_act else pre
        last[b] = m(rows[b, n:n + W - 1])
    return y, last


def conv_backward(x, w, dy, bias=None, silu_act=True, state=None, mag=False):
    """dict of dx, dw, dbias, dstate.  A magnitude counts the slope of silu as
    1 plus its sensitivity to the pre-activation's own magnitude."""
    x, w, dy, bias, state = map(_f, (x, w, dy, bias, state))
    m = np.abs if mag else (lambda v: v)
    B, L, E = x.shape
    W = w.shape[1]
    rows = _taps(x, state, W)
    drows = np.zeros_like(rows)
    dw, db = np.zeros_like(w), np.zeros(E)
    for t in range(L):
        tap = rows[:, t:t + W]
        pre = (tap * w.T).sum(1) + (0 if bias is None else bias)
        d = m(dy[:, t])
        if silu_act:
            size = (np.abs(tap * w.T)).sum(1) + (0 if bias is None else np.abs(bias))
            d = d * ((1.1 + size) if mag else dsilu(pre))
        db += d.sum(0)
        for k in range(W):
            dw[:, k] += (d * m(tap[:, k])).sum(0)
            drows[:, t + k] += d * m(w[:, k])
    return {"dx": drows[:, W - 1:], "dw": dw, "dbias": None if bias is None else db,
            "dstate": None if state is None else drows[:, :W - 1]}


def _rows_of(y, heads_first):
    return np.swapaxes(y, 1, 2) if heads_first else y  # [B, L, H, D]


def norm_gate(y, gate, w=None, eps=1e-5, gate_first=False, heads_first=True):
    """o [B, L, H*D]."""
    y, gate, w = map(_f, (y, gate, w))
    y = _rows_of(y, heads_first)
    act = silu(gate).reshape(y.shape)
    p = y * act if gate_first else y
    o = p / np.sqrt((p * p).mean(-1, keepdims=True) + eps)
    o = o if w is None else o * w
    return (o if gate_first else o * act).reshape(gate.shape)


def norm_gate_backward(y, gate, do, w=None, eps=1e-5, gate_first=False, heads_first=True, mag=False):
    """dict of dy (laid out as y), dgate, dw."""
    y, gate, do, w = map(_f, (y, gate, do, w))
    y = _rows_of(y, heads_first)
    g, do = gate.reshape(y.shape), do.reshape(y.shape)
    wv = np.ones(y.shape[2:]) if w is None else w
    m = np.abs if mag else (lambda v: v)
    act, dact = m(silu(g)), (dsilu_mag(g) if mag else dsilu(g))
    y, do, wv = m(y), m(do), m(wv)
    p = y * act if gate_first else y
    rstd = 1.0 / np.sqrt((p * p).mean(-1, keepdims=True) + eps)
    n = p * rstd
    dn = do * wv if gate_first else do * wv * act
    s = n * (dn * n).mean(-1, keepdims=True)
    dp = rstd * (dn + s if mag else dn - s)
    dw = (do * n if gate_first else do * n * act).sum((0, 1))
    dy, dg = (dp * act, dp * y * dact) if gate_first else (dp, do * n * wv * dact)
    return {"dy": np.swapaxes(dy, 1, 2) if heads_first else dy, "dgate": dg.reshape(gate.shape),
            "dw": None if w is None else dw}


def norm_residual(x, residual=None, w=None, scale=1.0, eps=1e-5):
    """(o, r)."""
    x, residual, w = map(_f, (x, residual, w))
    r = scale * x + (0 if residual is None else residual)
    o = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    return (o if w is None else o * w), r


def norm_residual_backward(r, do, w=None, dr=None, scale=1.0, eps=1e-5, mag=False):
    """dict of dresidual, dx, dw."""
    r, do, w, dr = map(_f, (r, do, w, dr))
    m = np.abs if mag else (lambda v: v)
    r, do = m(r), m(do)
    rstd = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    n = r * rstd
    dn = do if w is None else do * m(w)
    s = n * (dn * n).mean(-1, keepdims=True)
    d = rstd * (dn + s if mag else dn - s) + (0 if dr is None else m(dr))
    lead = tuple(range(r.ndim - 1))
    return {"dresidual": d, "dx": m(np.asarray(float(scale))) * d,
            "dw": None if w is None else (do * n).sum(lead)}
