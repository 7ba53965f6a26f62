"""Plain fp64 retention and beam selection (test infrastructure only).

Retention token by token: S_t = g S_(t-1) + k_t v_t^T, o_t = scale q_t^T S_t
("Attention-Free / Sub-Quadratic Architectures", "Evolution: add decay/gating":
RetNet's fixed decay, without feature map and normaliser), its gradients by
the adjoint recurrence U_t = g U_(t+1) + scale q_t do_t^T.  Arrays: q
[B][L][H][D], k, v [B][L][Hk][.], states [B][H][D][Dv], gamma [H].  mag: the
same sums over absolute values, the scale of their rounding errors.
"""
import numpy as np


def _f64(*arrays, mag=False):
    out = [None if a is None else np.asarray(a, dtype=np.float64) for a in arrays]
    return [None if a is None else np.abs(a) for a in out] if mag else out


def _shared(a, H):
    return np.repeat(a, H // a.shape[2], axis=2)


def _lens(lens, B, L):
    return np.full(B, L) if lens is None else np.clip(np.asarray(lens), 0, L)


def forward(q, k, v, gamma, scale=1.0, S0=None, lens=None, mag=False):
    """(o, S): rows of o behind a sequence's end are zero."""
    q, k, v, S0 = _f64(q, k, v, S0, mag=mag)
    scale = abs(scale) if mag else scale
    B, L, H, D = q.shape
    k, v = _shared(k, H), _shared(v, H)
    n = _lens(lens, B, L)
    g = np.asarray(gamma, dtype=np.float64)[None, :, None, None]
    S = np.zeros((B, H, D, v.shape[3])) if S0 is None else S0.copy()
    o = np.zeros((B, L, H, v.shape[3]))
    for t in range(L):
        live = t < n
        new = g * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        S = np.where(live[:, None, None, None], new, S)
        o[live, t] = scale * np.einsum("bhd,bhde->bhe", q[live, t], S[live])
    return o, S


def backward(q, k, v, do, gamma, scale=1.0, S0=None, dS=None, lens=None, mag=False):
    """(dq, dk, dv, dS0); dk and dv summed over the heads that share them."""
    q, k, v, do, S0, dS = _f64(q, k, v, do, S0, dS, mag=mag)
    scale = abs(scale) if mag else scale
    B, L, H, D = q.shape
    Hk, Dv = v.shape[2:]
    k, v = _shared(k, H), _shared(v, H)
    n = _lens(lens, B, L)
    g = np.asarray(gamma, dtype=np.float64)[None, :, None, None]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    S = np.zeros((B, H, D, Dv)) if S0 is None else S0.copy()
    for t in range(L):
        live = t < n
        S = np.where(live[:, None, None, None], g * S + k[:, t, :, :, None] * v[:, t, :, None, :], S)
        dq[live, t] = scale * np.einsum("bhde,bhe->bhd", S[live], do[live, t])
    U = np.zeros((B, H, D, Dv)) if dS is None else dS.copy()  # dL/dS behind token t
    for t in range(L - 1, -1, -1):
        live = (t < n)[:, None, None, None]
        U = np.where(live, U + scale * q[:, t, :, :, None] * do[:, t, :, None, :], U)
        dk[:, t] = np.where(live[..., 0], np.einsum("bhde,bhe->bhd", U, v[:, t]), 0)
        dv[:, t] = np.where(live[..., 0], np.einsum("bhde,bhd->bhe", U, k[:, t]), 0)
        U = np.where(live, g * U, U)
    share = lambda a: a.reshape(B, L, Hk, H // Hk, -1).sum(3)  # noqa: E731
    return dq, share(dk), share(dv), U


def select(logits, scores, n, finished=None, eos=None):
    """(scores, parents, tokens) [B][n] of the n best continuations."""
    B, K, V = logits.shape
    out = np.full((B, n), -np.inf), np.full((B, n), -1), np.full((B, n), -1)
    for b in range(B):
        cand = []
        for k in range(K):
            s = float(scores[b, k])
            if not np.isfinite(s):
                continue
            if finished is not None and finished[b, k]:
                cand.append((-s, k, eos))
                continue
            x = np.asarray(logits[b, k], dtype=np.float64)
            m = x.max() if not np.isnan(x).any() else np.nan
            if not np.isfinite(m):
                continue
            total = s + ((x - m) - np.log(np.exp(x - m).sum()))
            # candidates behind the n-th of their own row never enter
            keep = np.lexsort((np.arange(V), -x))[:n]
            cand += [(-total[i], k, int(i)) for i in keep if np.isfinite(x[i])]
        for r, (s, k, v) in enumerate(sorted(cand)[:n]):
            out[0][b, r], out[1][b, r], out[2][b, r] = -s, k, v
    return out
