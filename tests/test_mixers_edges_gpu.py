"""Edges of the selective scan family and of the calls around it on a GPU:
gates, decay rates and sizes at the ends of their ranges, calls behind a failed
one, and norm-wise bounds on what the element-wise ones leave loose.

Tolerances as in test_mixers_gpu.py; norm-wise ones are derived where they are
used."""
import numpy as np
import pytest
import torch

from helpers import record
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


@pytest.mark.parametrize("what", ["scan backward", "non-causal forward"])
def test_calls_behind_a_failed_workspace(la, what):
    """A call whose workspace is larger than the card reports it; the call
    behind it, whatever it is, checks its own launches and is not affected."""
    free, total = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB")
    a, more, d = scan_inputs(F32, (2, 90), 64, 16, 1, 23)
    args, dy, w = {**dev(a), **dev(more)}, d(2, 90, 64).cuda(), d.f(64, 4).cuda()
    one = {k: v[:, 0].contiguous() if k in ("x", "dt", "Bm", "Cm", "z") else v for k, v in args.items()}
    h, st, wn = torch.ones(2, 64, 16, device="cuda"), torch.ones(2, 3, 64, device="cuda"), w[:, 0].contiguous()
    q, gates, S = d(1, 2, 70, 64).cuda(), torch.full((1, 2, 70, 64), 0.5, device="cuda"), torch.ones(1, 2, 64, 64, device="cuda")
    q1 = q[:, :, 0].contiguous()
    small = [lambda: [la.forward_selective(**args)], lambda: la.backward_selective(**args, dy=dy)[:8],
             lambda: [la.decode_selective(**one, h=h.clone())], lambda: [la.forward_conv(dy, w)],
             lambda: la.backward_conv(dy, w, dy)[:2], lambda: [la.decode_conv(dy[:, 0], w, st.clone())],
             lambda: [la.forward_norm_gate(dy.view(2, 1, 90, 64), dy)], lambda: la.backward_norm_gate(dy.view(2, 1, 90, 64), dy, dy)[:2],
             lambda: la.forward_norm_residual(dy), lambda: la.backward_norm_residual(dy, dy, wn),
             lambda: [la.forward(q, q, q)], lambda: [la.forward(q, q, q, causal=False)], lambda: la.prefill_state(q, q),
             lambda: [la.forward_gated(q, q, q, gates)], lambda: la.backward(q, q, q, q),
             lambda: [la.decode_step(q1, q1, q1, S.clone(), S[..., 0].contiguous())], lambda: [dy + 1]]
    want = [f() for f in small]
    if what == "scan backward":  # two states of 64 fp32 per channel of 65536
        E, N = 65536, 64
        B = total // (E * N * 8) + 1000
        x, m = torch.empty(B, 1, E, dtype=BF16, device="cuda"), torch.empty(B, 1, 1, N, dtype=BF16, device="cuda")
        big = lambda: la.backward_selective(x, x, torch.empty(E, N, device="cuda"), m, m, x)  # noqa: E731
    else:  # a state of 128 x 129 fp32 per head, of one token each
        x = torch.empty(total // (256 * 128 * 129 * 4) + 1000, 256, 1, 128, device="cuda")
        big = lambda: la.forward(x, x, x, causal=False)  # noqa: E731
    for f, ref in zip(small, want):
        with pytest.raises(la.LinAttnError) as e:
            big()
        assert e.value.code == 3
        for u, v in zip(f(), ref):
            assert torch.equal(u, v)


@DT
@pytest.mark.parametrize("shape", [(1, 13, 64, 16, 1), (2, 70, 40, 8, 1), (1, 333, 264, 16, 3), (1, 333, 40, 64, 1)],
                         ids=lambda s: "x".join(map(str, s)))
def test_states_that_forget_at_once(la, dtype, shape):
    """Rates at the lowest fp32 value: a decay of zero at every token, and
    none at the rows behind a part's end, which hold no step."""
    B, L, E, N, G = shape
    a, more, d = scan_inputs(dtype, (B, L), E, N, G, L)
    a["A"][:, ::3] = torch.finfo(F32).min
    h0, dh, dy = d.f(B, E, N), d.f(B, E, N), d(B, L, E)
    K = 80 * (L + 4) + N
    y, h = la.forward_selective(**dev(a), **dev(more), h0=cuda(h0), return_state=True)
    (ry, rh), (my, mh) = scan_ref(a, more, True, h0=h0.numpy())
    close("scan lowest rates y", y, ry, my, K, dtype)
    close("scan lowest rates state", h, rh, mh, K, F32)
    got = la.backward_selective(**dev(a), dy=dy.cuda(), **dev(more), h0=cuda(h0), dh=cuda(dh))
    kw = {**host(a), **host(more), "dy": dy.float().numpy(), **host({"h0": h0, "dh": dh})}
    ref, mag = osel.scan_backward(**kw), osel.scan_backward(**kw, mag=True)
    for name, v in zip(GRADS, got):
        close("scan lowest rates " + name, v, ref[name], mag[name], 160 * (L + 8) + E + B * L, v.dtype)
    # an infinite rate is the same decay; a ragged batch ends inside a tile
    a["A"][:, ::3] = float("-inf")
    assert torch.equal(la.forward_selective(**dev(a), **dev(more), h0=cuda(h0)), y)
    lens = torch.full((B,), max(L - 5, 1), dtype=torch.int32)
    y, h = la.forward_selective(**dev(a), **dev(more), h0=cuda(h0), lens=cuda(lens), out=torch.zeros_like(y), return_state=True)
    (ry, rh), (my, mh) = scan_ref(a, more, True, h0=h0.numpy(), lens=lens.numpy())
    close("scan infinite rates y", y, ry, my, K, dtype)
    close("scan infinite rates state", h, rh, mh, K, F32)
    one = {k: v[:, 0] if k in ("x", "dt", "Bm", "Cm", "z") else v for k, v in {**a, **more}.items()}
    hs = cuda(h0).clone()
    y = la.decode_selective(**dev(one), h=hs)
    (ry, rh), (my, mh) = [osel.scan_step(**host(one), h=h0.numpy(), mag=m) for m in (False, True)]
    close("scan infinite rates step y", y, ry, my, 80 * 5 + N, dtype)
    close("scan infinite rates step state", hs, rh, mh, 80 * 5, F32)


def close_in_norm(name, got, ref, tol, dtype):
    """||got - ref|| against tol and half a step of the output's type, both of
    ||ref||."""
    rel = np.linalg.norm(n64(got) - ref) / np.linalg.norm(ref)
    bound = tol + (0 if dtype == F32 else torch.finfo(dtype).eps / 2)
    record(f"{name} {str(dtype)[6:]} (norm)", rel, bound)
    assert rel <= bound, f"{name}: {rel}, bound {bound}"


# Several parts, groups, channel tiles, all numbers of states.
MANY_PARTS = [(2, 400, 264, 8, 1), (1, 700, 528, 16, 2), (1, 500, 264, 32, 1), (2, 300, 72, 64, 1), (3, 1500, 16, 16, 1)]


@DT
@pytest.mark.parametrize("shape", MANY_PARTS, ids=lambda s: "x".join(map(str, s)))
def test_many_parts_in_norm(la, dtype, shape):
    """The scan over many parts, norm-wise: fewer bits in a record or a
    checkpoint show here, where the element bounds are far wider.

    A state remembers 1 / (dt |A|) tokens, at most about 1 / (0.01 x 0.05) =
    2000 with these inputs, and takes about 5.5 roundings a token (the
    exponential 4, the product and sum 1.5; the exponent of a state that
    remembers long is near zero).  Independent roundings add up as
    sqrt(2000) x 5.5 = 250 of 2^-24: 1.5e-5, 2e-5 with what stands around the
    recurrence.  Gradients take a second recurrence: 4e-5.  A record in bf16
    would be off by 2^-9 / sqrt(3) = 1.1e-3 of itself."""
    B, L, E, N, G = shape
    a, more, d = scan_inputs(dtype, (B, L), E, N, G, 3 * L + N)
    h0, dh, dy = d.f(B, E, N), d.f(B, E, N), d(B, L, E)
    p = {**dev(a), **dev(more), "h0": cuda(h0)}
    y, h = la.forward_selective(**p, return_state=True)
    hp = {**host(a), **host(more), "h0": h0.numpy()}
    ry, rh = osel.scan(**hp)
    close_in_norm("scan y", y, ry, 2e-5, dtype)
    close_in_norm("scan state", h, rh, 2e-5, F32)
    lens = (torch.rand(B, generator=d.g) * L).to(torch.int32) + 1
    y, h = la.forward_selective(**p, lens=cuda(lens), out=torch.zeros_like(y), return_state=True)
    ry, rh = osel.scan(**hp, lens=lens.numpy())
    close_in_norm("scan ragged y", y, ry, 2e-5, dtype)
    close_in_norm("scan ragged state", h, rh, 2e-5, F32)
    got = la.backward_selective(**p, dy=dy.cuda(), dh=cuda(dh))
    ref = osel.scan_backward(**hp, dy=dy.float().numpy(), dh=dh.numpy())
    for name, v in zip(GRADS, got):
        close_in_norm("scan " + name, v, ref[name], 4e-5, v.dtype)


@DT
@pytest.mark.parametrize("shape", [(3, 75, 64, 16, 1), (2, 300, 72, 8, 1), (2, 130, 40, 64, 1)], ids=lambda s: "x".join(map(str, s)))
def test_backward_of_a_padded_batch(la, dtype, shape):
    """Rows of padding with a raw step of -inf (softplus: a step of zero) and
    zero rows of dy: every sequence gets the gradients that it has alone, also
    through its final state, and the padding none but dz = 0."""
    B, L, E, N, G = shape
    a, more, d = scan_inputs(dtype, (B, L), E, N, G, 31)
    h0, dh, dy = d.f(B, E, N), d.f(B, E, N), d(B, L, E)
    lens = [L - 1 - (b * L) // (B + 1) for b in range(B)]
    for b, n in enumerate(lens):
        a["dt"][b, n:] = float("-inf")
        dy[b, n:] = 0
    got = la.backward_selective(**dev(a), dy=dy.cuda(), **dev(more), h0=cuda(h0), dh=cuda(dh))
    parts = []
    for b, n in enumerate(lens):
        one = {k: v[b:b + 1, :n] if k in ("x", "dt", "Bm", "Cm", "z") else v for k, v in {**a, **more}.items()}
        kw = {**host(one), "dy": dy[b:b + 1, :n].float().numpy(), **host({"h0": h0[b:b + 1], "dh": dh[b:b + 1]})}
        parts.append([osel.scan_backward(**kw, mag=m) for m in (False, True)])
    K = 160 * (L + 8) + E + B * L
    for name, v in zip(GRADS, got):
        if name in ("dA", "dD", "ddt_bias"):  # sums over the batch
            close("scan padded " + name, v, sum(r[name] for r, _ in parts), sum(m[name] for _, m in parts), K, F32)
            continue
        for b, (ref, mag) in enumerate(parts):
            own = v[b:b + 1] if name == "dh0" else v[b:b + 1, :lens[b]]
            close("scan padded " + name, own, ref[name], mag[name], K, v.dtype)
            if name != "dh0":
                assert (v[b, lens[b]:] == 0).all(), name
