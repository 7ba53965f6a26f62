"""Edges of the selective scan family and of the calls around it on a GPU:
gates, decay rates and sizes at the ends of their ranges, calls behind a failed
one, and norm-wise bounds on what the element-wise ones leave loose.

Tolerances as in test_mixers_gpu.py; norm-wise ones are derived where they are
used."""
import numpy as np
import pytest
import torch

from oracle import selective as osel
from test_mixers_gpu import BF16, DT, F32, Draw, close, cuda, dev, host, la, n64, scan_inputs, scan_ref  # noqa: F401

pytestmark = pytest.mark.gpu

GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")


@DT
def test_gates_of_the_lowest_value(la, dtype):
    """silu of the type's lowest value is zero: outputs and slopes there are
    zero, in every form of the scan, also where y is large."""
    B, L, E, N = 2, 37, 64, 16
    a, more, d = scan_inputs(dtype, (B, L), E, N, 1, 21)
    a["x"] *= 8
    low = torch.finfo(dtype).min
    more["z"][:, ::3] = low
    more["z"][:, :, 5] = low
    shut = (more["z"] == low).cuda()
    y, h = la.forward_selective(**dev(a), **dev(more), return_state=True)
    (ry, rh), (my, mh) = scan_ref(a, more, True)
    assert (y[shut] == 0).all()
    close("scan low gates y", y, ry, my, 80 * (L + 4) + N, dtype)
    close("scan low gates state", h, rh, mh, 80 * (L + 4) + N, F32)
    one = {k: v[:, 0] if k in ("x", "dt", "Bm", "Cm", "z") else v for k, v in {**a, **more}.items()}
    h = d.f(B, E, N)
    y = la.decode_selective(**dev(one), h=cuda(h).clone())
    (ry, _), (my, _) = [osel.scan_step(**host(one), h=h.numpy(), mag=m) for m in (False, True)]
    assert (y == 0).all()
    close("scan low gates step y", y, ry, my, 80 * 5 + N, dtype)
    dy = d(B, L, E)
    got = la.backward_selective(**dev(a), dy=dy.cuda(), **dev(more))
    kw = {**host(a), **host(more), "dy": dy.float().numpy()}
    ref, mag = osel.scan_backward(**kw), osel.scan_backward(**kw, mag=True)
    assert (got[6][shut] == 0).all()
    for name, v in zip(GRADS[:8], got):
        close("scan low gates " + name, v, ref[name], mag[name], 160 * (L + 8) + E + B * L, v.dtype)


@DT
def test_infinite_gates(la, dtype):
    """An infinite gate gives what the formula gives (y inf; inf times 0), in
    its own place and channel, the same for a prompt and a token."""
    B, L, E, N = 2, 37, 64, 16
    a, more, d = scan_inputs(dtype, (B, L), E, N, 1, 22)
    clean = {**dev(a), **dev(more)}
    bad = {**clean, "z": clean["z"].clone()}
    at = [(0, 3, 7), (1, 36, 9)]
    bad["z"][at[0]], bad["z"][at[1]] = float("inf"), float("-inf")
    y0, y = la.forward_selective(**clean), la.forward_selective(**bad)
    assert torch.isinf(y[at[0]]) and torch.isnan(y[at[1]])
    assert torch.sign(y[at[0]]) == torch.sign(y0[at[0]]) * torch.sign(clean["z"][at[0]])
    for i in at:
        y[i] = y0[i]
    assert torch.equal(y, y0)
    for (b, t, e), inf in zip(at, (True, False)):
        one = {k: v[:, t].contiguous() if k in ("x", "dt", "Bm", "Cm", "z") else v for k, v in bad.items()}
        ys = la.decode_selective(**one, h=torch.ones(B, E, N, device="cuda"))
        assert torch.isinf(ys[b, e]) if inf else torch.isnan(ys[b, e])
        assert int(torch.isfinite(ys).sum()) == B * E - 1
    dy = d(B, L, E).cuda()
    g0, g = la.backward_selective(**clean, dy=dy), la.backward_selective(**bad, dy=dy)
    other = torch.ones(E, dtype=torch.bool)
    other[[7, 9]] = False
    for i in (0, 1, 6):  # dx, ddt, dz of the other channels
        assert torch.equal(g[i][..., other], g0[i][..., other])
    for i in (2, 5, 7):  # dA, dD, d(dt_bias)
        assert torch.equal(g[i][other], g0[i][other])
