"""GPU parity of the selective state space scan, its short convolution and the
norms around a block against the fp64 oracle.

Tolerances, element by element: half a step of the output's type, relative to
the value, plus K x 2^-24 x the element's magnitude (the same sums over
absolute values, from the oracle), where K counts the fp32 roundings on the
longest path to the output, for values that the oracle gets as the kernel does:

  scan     a token adds to a state the errors of softplus (6 x 2^-24: its
           interpolant is off by 3.2e-7), of the exponential (4) and of its
           argument (|dt A| up to 8 here, times 6 + 2), the product and the
           sum: at most 80 per token, linear in the tokens walked;
  scan,    the adjoint adds as much again, and the sums over channels and
  backward tokens one per term: 160 (L + 8) + E + B L;
  conv     W products and sums, the activation (8): 16; its sums one per token;
  norms    D / 8 sums in a lane and their tree, the root, the products: D / 8 + 32,
           and one per row for the weight's gradient.
"""
import numpy as np
import pytest
import torch

from helpers import record
from oracle import selective as osel

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DT = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kernelized_sequence_mixing_gb300 import build
    build.build()
    import kernelized_sequence_mixing_gb300 as m
    return m


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def close(name, got, ref, mag, K, dtype):
    got = n64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), name
    if not got.size:
        return
    # results below the type's normal range may be flushed
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + K * 2.0 ** -24 * np.asarray(mag) + 1e-37
    worst = float((np.abs(got - ref) / tol).max())
    record(f"{name} {str(dtype)[6:]} (share of its bound)", worst, 1)
    assert worst <= 1, f"{name}: {worst} times its bound"


class Draw:
    def __init__(self, seed, dtype):
        self.g = torch.Generator().manual_seed(seed)
        self.t = dtype

    def __call__(self, *shape, scale=1.0, dtype=None):
        return (torch.randn(shape, generator=self.g) * scale).to(dtype or self.t)

    def f(self, *shape, scale=1.0):
        return self(*shape, scale=scale, dtype=F32)


def cuda(t):
    return None if t is None else t.cuda()


def scan_inputs(dtype, lead, E, N, G, seed, bare=False):
    d = Draw(seed, dtype)
    a = {"x": d(*lead, E), "dt": d(*lead, E), "A": -torch.rand(E, N, generator=d.g) * 4 - 0.05,
         "Bm": d(*lead, G, N), "Cm": d(*lead, G, N)}
    # steps of about 0.003 to 1
    more = {"D": d.f(E), "z": d(*lead, E), "dt_bias": d.f(E) - 3.0}
    if bare:
        more = {k: None for k in more}
        a["dt"] = (torch.rand(*lead, E, generator=d.g) * 0.5).to(dtype)
    return a, more, d


def host(d):
    return {k: None if v is None else v.float().numpy() for k, v in d.items()}


def dev(d):
    return {k: cuda(v) for k, v in d.items()}


def scan_ref(a, more, sp, **kw):
    ha, hm = host(a), host(more)
    return [osel.scan(**ha, **hm, softplus_dt=sp, mag=m, **kw) for m in (False, True)]


# (B, L, E, N, G): one token, odd lengths, parts of every state size (two and
# more), channel tails, groups
SCANS = [
    (1, 1, 8, 16, 1), (2, 3, 72, 8, 1), (1, 17, 136, 16, 1), (3, 65, 64, 32, 2), (1, 63, 40, 64, 1),
    (1, 333, 264, 16, 1), (2, 300, 48, 8, 2), (1, 520, 96, 64, 4), (1, 1000, 16, 32, 1),
    (5, 2, 512, 16, 4), (1, 2800, 64, 8, 8), (2, 97, 40, 64, 1),
]
sid = lambda s: "x".join(map(str, s))  # noqa: E731


@DT
@pytest.mark.parametrize("bare", [False, True], ids=["full", "bare"])
@pytest.mark.parametrize("shape", SCANS, ids=sid)
def test_scan(la, dtype, bare, shape):
    B, L, E, N, G = shape
    a, more, d = scan_inputs(dtype, (B, L), E, N, G, L + E, bare)
    h0 = None if bare else d.f(B, E, N)
    y, h = la.forward_selective(**dev(a), **dev(more), softplus=not bare, h0=cuda(h0),
                                return_state=True)
    (ry, rh), (my, mh) = scan_ref(a, more, not bare, h0=None if bare else h0.numpy())
    K = 80 * (L + 4) + N
    close("scan y", y, ry, my, K, dtype)
    close("scan state", h, rh, mh, K, F32)
    y2 = la.forward_selective(**dev(a), **dev(more), softplus=not bare, h0=cuda(h0))
    assert torch.equal(y, y2)


@DT
def test_scan_ragged(la, dtype):
    """Rows behind a sequence's end: not read (NaN there), not written."""
    B, L, E, N = 6, 400, 64, 16
    a, more, d = scan_inputs(dtype, (B, L), E, N, 1, 5)
    lens = torch.tensor([400, 0, 1, 257, 399, -3], dtype=torch.int32)
    h0 = d.f(B, E, N)
    for k, t in [(k, a[k]) for k in ("x", "dt", "Bm", "Cm")] + [("z", more["z"])]:
        for b in range(B):
            t[b, max(int(lens[b]), 0):] = float("nan")
    out = torch.full((B, L, E), -3.0, dtype=dtype).cuda()
    y, h = la.forward_selective(**dev(a), **dev(more), h0=cuda(h0), lens=cuda(lens), out=out,
                                return_state=True)
    kept = np.full((B, L, E), -3.0)
    (ry, rh), (my, mh) = scan_ref(a, more, True, h0=h0.numpy(), lens=lens.numpy(), out=kept)
    close("scan ragged y", y, ry, my, 80 * (L + 4), dtype)
    close("scan ragged state", h, rh, mh, 80 * (L + 4), F32)
    for b in range(B):
        assert (y[b, max(int(lens[b]), 0):] == -3.0).all()
    # the same rows alone give the same values bit for bit up to the part split
    long = torch.tensor([L + 7] * B, dtype=torch.int32).cuda()  # clamped to L
    full = {k: torch.nan_to_num(v) for k, v in a.items()}
    fm = {k: torch.nan_to_num(v) for k, v in more.items()}
    assert torch.equal(la.forward_selective(**dev(full), **dev(fm), lens=long),
                       la.forward_selective(**dev(full), **dev(fm)))


@DT
@pytest.mark.parametrize("B,L,E,N", [(3, 700, 64, 16), (40, 500, 8, 8), (100, 97, 16, 64), (2, 6000, 40, 32)])
def test_scan_ragged_parts(la, dtype, B, L, E, N):
    """Batches whose parts are laid out by the lengths: more sequences than a
    warp has lanes, empty ones first and last, one long among short ones."""
    a, more, d = scan_inputs(dtype, (B, L), E, N, 1, B)
    lens = (torch.rand(B, generator=d.g) ** 3 * (L + 20)).to(torch.int32)
    lens[0], lens[-1], lens[B // 2] = 0, -1, L
    h0 = d.f(B, E, N)
    y, h = la.forward_selective(**dev(a), **dev(more), h0=cuda(h0), lens=cuda(lens), return_state=True)
    (ry, rh), (my, mh) = scan_ref(a, more, True, h0=h0.numpy(), lens=lens.numpy())
    rows = np.arange(L)[None, :] < lens.numpy()[:, None]
    close("scan ragged y", torch.where(torch.from_numpy(rows)[..., None].cuda(), y, 0), np.where(rows[..., None], ry, 0),
          np.where(rows[..., None], my, 0), 80 * (L + 4), dtype)
    close("scan ragged state", h, rh, mh, 80 * (L + 4), F32)
    none = lens <= 0
    assert torch.equal(h.cpu()[none], h0[none])


@DT
@pytest.mark.parametrize("shape", [(1, 8, 16, 1), (3, 72, 8, 1), (2, 64, 32, 2), (65, 96, 64, 4),
                                   (256, 4096, 16, 1)], ids=sid)
def test_scan_step(la, dtype, shape):
    B, E, N, G = shape
    a, more, d = scan_inputs(dtype, (B,), E, N, G, B)
    h = d.f(B, E, N)
    hc = cuda(h).clone()
    y = la.decode_selective(**dev(a), h=hc, **dev(more))
    ha, hm = host(a), host(more)
    (ry, rh), (my, mh) = [osel.scan_step(**ha, h=h.numpy(), **hm, mag=m) for m in (False, True)]
    close("scan step y", y, ry, my, 80 * 5 + N, dtype)
    close("scan step state", hc, rh, mh, 80 * 5, F32)


@DT
@pytest.mark.parametrize("start", [False, True], ids=["zero", "state"])
@pytest.mark.parametrize("shape", SCANS, ids=sid)
def test_scan_backward(la, dtype, start, shape):
    B, L, E, N, G = shape
    bare = not start and L % 2 == 1
    a, more, d = scan_inputs(dtype, (B, L), E, N, G, 7 * L + E, bare)
    dy = d(B, L, E)
    h0, dh = (d.f(B, E, N), d.f(B, E, N)) if start else (None, None)
    got = la.backward_selective(**dev(a), dy=dy.cuda(), **dev(more), softplus=not bare, h0=cuda(h0),
                                dh=cuda(dh))
    kw = {**host(a), **host(more), "dy": dy.float().numpy(), "softplus_dt": not bare,
          **host({"h0": h0, "dh": dh})}
    ref, mag = osel.scan_backward(**kw), osel.scan_backward(**kw, mag=True)
    K = 160 * (L + 8) + E + B * L
    for name, v in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0"), got):
        assert (v is None) == (ref[name] is None), name
        if v is not None:
            close("scan " + name, v, ref[name], mag[name], K, v.dtype)
    again = la.backward_selective(**dev(a), dy=dy.cuda(), **dev(more), softplus=not bare,
                                  h0=cuda(h0), dh=cuda(dh))
    for u, v in zip(got, again):  # fixed orders of summation
        assert u is None or torch.equal(u, v)


def test_scan_gradients_by_differences(la):
    """The kernel's own forward, in fp32, by central differences: the change
    of sum(y dy) along random directions of all inputs at once."""
    B, L, E, N, G = 1, 70, 16, 8, 2
    a, more, d = scan_inputs(F32, (B, L), E, N, G, 3)
    dy, h0, dh = d(B, L, E), d.f(B, E, N), d.f(B, E, N)
    p = {**dev(a), **dev(more), "h0": h0.cuda()}
    got = dict(zip(("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0"),
                   la.backward_selective(**p, dy=dy.cuda(), dh=dh.cuda())))

    def loss(q):
        y, h = la.forward_selective(**q, return_state=True)
        return float((y.double() * dy.cuda().double()).sum() + (h.double() * dh.cuda().double()).sum())

    for seed in range(4):
        dr = Draw(100 + seed, F32)
        v = {k: dr(*t.shape, scale=0.05 if k == "A" else 1.0).cuda() for k, t in p.items()}
        s = 2.0 ** -9
        num = (loss({k: p[k] + s * v[k] for k in p}) - loss({k: p[k] - s * v[k] for k in p})) / (2 * s)
        ana = sum(float((got[k].double() * v[k].double()).sum()) for k in p)
        size = sum(float((got[k].double() * v[k].double()).abs().sum()) for k in p)
        # the third-order term is about s^2 of the size, the outputs' rounding 2^-24 / s of it
        assert abs(num - ana) <= (32 * s * s + 2.0 ** -24 / s * 32) * size


CONVS = [(1, 1, 8, 2), (2, 2, 24, 4), (3, 33, 72, 3), (1, 47, 264, 4), (2, 257, 512, 2), (1, 1030, 64, 4)]


@DT
@pytest.mark.parametrize("full", [False, True], ids=["bare", "full"])
@pytest.mark.parametrize("shape", CONVS, ids=sid)
def test_conv(la, dtype, full, shape):
    B, L, E, W = shape
    d = Draw(L, dtype)
    x, w = d(B, L, E), d.f(E, W)
    bias, state = (d.f(E), d(B, W - 1, E)) if full else (None, None)
    y, last = la.forward_conv(x.cuda(), w.cuda(), cuda(bias), silu=full, state=cuda(state),
                              return_state=True)
    kw = host({"x": x, "w": w, "bias": bias, "state": state})
    (ry, rl), (my, _) = [osel.conv(**kw, silu_act=full, mag=m) for m in (False, True)]
    close("conv y", y, ry, my, 16, dtype)
    assert np.array_equal(n64(last), rl)
    # token by token from the same state
    st = torch.zeros(B, W - 1, E, dtype=dtype).cuda() if state is None else state.cuda()
    for t in range(min(L, 5)):
        yt = la.decode_conv(x[:, t].contiguous().cuda(), w.cuda(), st, cuda(bias), silu=full)
        close("conv step y", yt, ry[:, t], my[:, t], 16, dtype)


@DT
def test_conv_ragged(la, dtype):
    B, L, E, W = 6, 50, 40, 4
    d = Draw(3, dtype)
    x, w, bias, state = d(B, L, E), d.f(E, W), d.f(E), d(B, W - 1, E)
    lens = torch.tensor([50, 0, 1, 2, 17, -1], dtype=torch.int32)
    for b in range(B):
        x[b, max(int(lens[b]), 0):] = float("nan")
    out = torch.full((B, L, E), -3.0, dtype=dtype).cuda()
    y, last = la.forward_conv(x.cuda(), w.cuda(), bias.cuda(), state=state.cuda(), lens=lens.cuda(),
                              out=out, return_state=True)
    kw = host({"x": x, "w": w, "bias": bias, "state": state})
    with np.errstate(invalid="ignore"):
        (ry, rl), (my, _) = [osel.conv(**kw, lens=lens.numpy(), out=np.full((B, L, E), -3.0), mag=m)
                             for m in (False, True)]
    close("conv ragged y", y, ry, np.abs(my), 16, dtype)
    assert np.array_equal(n64(last), rl)


@DT
@pytest.mark.parametrize("full", [False, True], ids=["bare", "full"])
@pytest.mark.parametrize("shape", CONVS, ids=sid)
def test_conv_backward(la, dtype, full, shape):
    B, L, E, W = shape
    d = Draw(L + 1, dtype)
    x, w, dy = d(B, L, E), d.f(E, W), d(B, L, E)
    bias, state = (d.f(E), d(B, W - 1, E)) if full else (None, None)
    got = la.backward_conv(x.cuda(), w.cuda(), dy.cuda(), cuda(bias), silu=full, state=cuda(state))
    kw = host({"x": x, "w": w, "dy": dy, "bias": bias, "state": state})
    ref, mag = [osel.conv_backward(**kw, silu_act=full, mag=m) for m in (False, True)]
    for name, v in zip(("dx", "dw", "dbias", "dstate"), got):
        assert (v is None) == (ref[name] is None), name
        if v is not None:
            close("conv " + name, v, ref[name], mag[name], 32 + (0 if name in ("dx", "dstate") else B * L),
                  v.dtype)


# (B, H, L, D): widths on both sides of every change of lanes
GATES = [(1, 1, 1, 8), (2, 3, 5, 32), (1, 2, 33, 40), (2, 4, 17, 64), (1, 3, 70, 128), (2, 1, 9, 136),
         (1, 2, 7, 256), (1, 2, 3, 264), (1, 1, 19, 512), (1, 2, 5, 1000), (2, 1, 3, 1032),
         (1, 1, 4, 2048), (1, 1, 2, 2056), (1, 1, 3, 4096), (1, 1, 2, 8192)]
MODES = pytest.mark.parametrize("mode", [(False, True), (True, True), (False, False), (True, False)],
                                ids=["after-heads", "first-heads", "after-tokens", "first-tokens"])


@DT
@MODES
@pytest.mark.parametrize("shape", GATES, ids=sid)
def test_norm_gate(la, dtype, mode, shape):
    B, H, L, D = shape
    gate_first, heads_first = mode
    d = Draw(D, dtype)
    y = d(B, H, L, D) if heads_first else d(B, L, H, D)
    gate, w, do = d(B, L, H * D), d.f(H, D), d(B, L, H * D)
    if D == 64:
        y[0, 0, 0] = 0  # a row of zeros
    if D == 40:
        w = None
    kw = {"eps": 1e-5, "gate_first": gate_first, "heads_first": heads_first}
    o = la.forward_norm_gate(y.cuda(), gate.cuda(), cuda(w), **kw)
    h = host({"y": y, "gate": gate, "w": w})
    ref = osel.norm_gate(**h, **kw)
    K = D / 8 + 32
    close("norm gate o", o, ref, np.abs(ref), K, dtype)
    got = la.backward_norm_gate(y.cuda(), gate.cuda(), do.cuda(), cuda(w), **kw)
    ref, mag = [osel.norm_gate_backward(**h, do=do.float().numpy(), **kw, mag=m) for m in (False, True)]
    for name, v in zip(("dy", "dgate", "dw"), got):
        assert (v is None) == (ref[name] is None), name
        if v is not None:
            close("norm gate " + name, v, ref[name], mag[name], K + (B * L if name == "dw" else 0), v.dtype)


@DT
@pytest.mark.parametrize("full", [False, True], ids=["bare", "full"])
@pytest.mark.parametrize("shape", [(1, 8), (7, 72), (2, 3, 256), (33, 1024), (5, 1032), (700, 2048),
                                   (3, 4104), (2, 8192)], ids=sid)
def test_norm_residual(la, dtype, full, shape):
    E = shape[-1]
    d = Draw(E, dtype)
    x, res, do = d(*shape), d(*shape, scale=2.0), d(*shape)
    w, dr, scale = (d.f(E), d(*shape), 0.25) if full else (None, None, 1.0)
    if not full:
        res = None
    o, r = la.forward_norm_residual(x.cuda(), cuda(res), cuda(w), scale=scale)
    h = host({"x": x, "residual": res, "w": w})
    ro, rr = osel.norm_residual(**h, scale=scale)
    K = E / 8 + 32
    size = scale * np.abs(n64(x)) + (0 if res is None else np.abs(n64(res)))
    close("norm residual r", r, rr, size, 2, dtype)
    # r's own error (2 roundings of its terms' size) passes through the norm
    rstd = np.abs(1 / np.sqrt((rr * rr).mean(-1, keepdims=True) + 1e-5)) * (1 if w is None else np.abs(n64(w)))
    close("norm residual o", o, ro, size * rstd, K, dtype)
    got = la.backward_norm_residual(r, do.cuda(), cuda(w), cuda(dr), scale=scale)
    hb = {"r": r.float().cpu().numpy(), **host({"do": do, "w": w, "dr": dr})}
    ref, mag = [osel.norm_residual_backward(**hb, scale=scale, mag=m) for m in (False, True)]
    rows = int(np.prod(shape[:-1]))
    for name, v in zip(("dresidual", "dx", "dw"), got):
        assert (v is None) == (ref[name] is None), name
        if v is not None:
            close("norm residual " + name, v, ref[name], mag[name], K + (rows if name == "dw" else 0), v.dtype)
    assert full or got[1] is got[0]


@DT
def test_strided_inputs(la, dtype):
    """Slices of a projection's output, read in place: the same bits as dense
    copies."""
    B, L, E, N, G = 2, 150, 64, 16, 2
    a, more, d = scan_inputs(dtype, (B, L), E, N, G, 9)
    xz = torch.cat((a["x"], more["z"]), -1).cuda()
    bc = torch.stack((a["Bm"], a["Cm"]), 2).cuda()
    wide = torch.cat((a["dt"], a["dt"]), -1).cuda()
    x, z, dt = xz[..., :E], xz[..., E:], wide[..., E:]
    Bm, Cm = bc[:, :, 0], bc[:, :, 1]
    da, dm = dev(a), dev(more)
    s = {**da, **dm, "x": x, "z": z, "dt": dt, "Bm": Bm, "Cm": Cm}
    assert not x.is_contiguous() and not Cm.is_contiguous()
    assert torch.equal(la.forward_selective(**s), la.forward_selective(**da, **dm))
    dy = d(B, L, E).cuda()
    for u, v in zip(la.backward_selective(**s, dy=dy), la.backward_selective(**da, **dm, dy=dy)):
        assert u is None or torch.equal(u, v)
    w = d.f(E, 4).cuda()
    assert torch.equal(la.forward_conv(x, w), la.forward_conv(da["x"], w))
    for u, v in zip(la.backward_conv(x, w, dy), la.backward_conv(da["x"], w, dy)):
        assert u is None or torch.equal(u, v)
    one = {k: (v[:, 0] if k in ("x", "z", "dt", "Bm", "Cm") else v) for k, v in s.items()}
    dense = {k: v.contiguous() for k, v in one.items()}
    h = [torch.zeros(B, E, N, device="cuda") for _ in range(2)]
    assert torch.equal(la.decode_selective(**one, h=h[0]), la.decode_selective(**dense, h=h[1]))
    st = [torch.zeros(B, 3, E, dtype=dtype, device="cuda") for _ in range(2)]
    assert torch.equal(la.decode_conv(one["x"], w, st[0]), la.decode_conv(dense["x"], w, st[1]))


def test_empty_calls(la):
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    E, N = 16, 8
    A, h0 = -f(E, N), f(2, E, N) * 3
    y, h = la.forward_selective(f(2, 0, E), f(2, 0, E), A, f(2, 0, 1, N), f(2, 0, 1, N), h0=h0,
                                return_state=True)
    assert y.shape == (2, 0, E) and torch.equal(h, h0)
    got = la.backward_selective(f(2, 0, E), f(2, 0, E), A, f(2, 0, 1, N), f(2, 0, 1, N), f(2, 0, E),
                                D=f(E), dt_bias=f(E), h0=h0, dh=h0)
    assert (got[2] == 0).all() and (got[5] == 0).all() and (got[7] == 0).all()
    assert torch.equal(got[8], h0)
    got = la.backward_selective(f(0, 4, E), f(0, 4, E), A, f(0, 4, 1, N), f(0, 4, 1, N), f(0, 4, E), D=f(E))
    assert (got[2] == 0).all() and (got[5] == 0).all()
    w = f(E, 4)
    y, st = la.forward_conv(f(2, 0, E), w, state=f(2, 3, E), return_state=True)
    assert y.shape == (2, 0, E) and (st == 1).all()
    y, st = la.forward_conv(f(2, 0, E), w, return_state=True)
    assert (st == 0).all()
    dx, dw, db, dst = la.backward_conv(f(2, 0, E), w, f(2, 0, E), f(E), state=f(2, 3, E))
    assert (dw == 0).all() and (db == 0).all() and (dst == 0).all()
    dw = la.backward_norm_gate(f(1, 2, 0, 8), f(1, 0, 16), f(1, 0, 16), f(2, 8))[2]
    assert dw.shape == (2, 8) and (dw == 0).all()
    assert (la.backward_norm_residual(f(0, 8), f(0, 8), f(8))[2] == 0).all()
    assert la.decode_selective(f(0, E), f(0, E), A, f(0, 1, N), f(0, 1, N), f(0, E, N)).shape == (0, E)


def test_special_values(la):
    """Steps from a wide range of raw values, decays that reach zero, a NaN
    that stays in its channel and after its token."""
    B, L, E, N = 1, 40, 32, 16
    a, more, d = scan_inputs(F32, (B, L), E, N, 1, 2)
    a["dt"] = torch.linspace(-90, 60, L * E).reshape(1, L, E)
    more["dt_bias"] = None
    y, h = la.forward_selective(**dev(a), **dev(more), return_state=True)
    (ry, rh), (my, mh) = scan_ref(a, more, True)
    # |dt A| up to 250: the exponent's rounding counts that often
    close("scan wide steps y", y, ry, my, 80 * 250, F32)
    close("scan wide steps state", h, rh, mh, 80 * 250, F32)
    a, more, d = scan_inputs(F32, (B, L), E, N, 1, 2)
    clean = la.forward_selective(**dev(a), **dev(more))
    a["x"][0, 7, 5] = float("nan")
    bad = la.forward_selective(**dev(a), **dev(more))
    assert torch.isnan(bad[0, 7:, 5]).all()
    bad[0, 7:, 5] = clean[0, 7:, 5]
    assert torch.equal(bad, clean)


@DT
@pytest.mark.parametrize("gate_first", [False, True], ids=["after", "first"])
def test_norms_of_extreme_rows(la, dtype, gate_first):
    """Rows whose rstd cubed leaves the fp32 range: zeros and 2^-45 under a
    small eps, 2^60 at the other end.  The same roundings as other rows."""
    eps, D = 2.0 ** -100, 64
    d = Draw(11, dtype)
    size = torch.tensor([0, 2.0 ** -45, 2.0 ** 60, 1.0])[:, None]
    y = (d(1, 2, 4, D, dtype=F32) * size).to(dtype)
    gate, w, do = d(1, 4, 2 * D), d.f(2, D), d(1, 4, 2 * D)
    kw = {"eps": eps, "gate_first": gate_first, "heads_first": True}
    h = host({"y": y, "gate": gate, "w": w})
    K = D / 8 + 32
    ref = osel.norm_gate(**h, **kw)
    close("norm gate extremes o", la.forward_norm_gate(y.cuda(), gate.cuda(), w.cuda(), **kw), ref, np.abs(ref), K, dtype)
    got = la.backward_norm_gate(y.cuda(), gate.cuda(), do.cuda(), w.cuda(), **kw)
    ref, mag = [osel.norm_gate_backward(**h, do=do.float().numpy(), **kw, mag=m) for m in (False, True)]
    for name, v in zip(("dy", "dgate", "dw"), got):
        close("norm gate extremes " + name, v, ref[name], mag[name], K + (4 if name == "dw" else 0), v.dtype)
    r, do, w = y[0, 0].contiguous(), d(4, D), d.f(D)
    got = la.backward_norm_residual(r.cuda(), do.cuda(), w.cuda(), eps=eps)
    hb = host({"r": r, "do": do, "w": w, "dr": None})
    ref, mag = [osel.norm_residual_backward(**hb, scale=1.0, eps=eps, mag=m) for m in (False, True)]
    for name, v in zip(("dresidual", "dx", "dw"), got):
        close("norm residual extremes " + name, v, ref[name], mag[name], K + (4 if name == "dw" else 0), v.dtype)


def test_one_tensor_as_two_inputs(la):
    """Inputs are only read: a tensor may stand for two of them."""
    d = Draw(12, BF16)
    x, bc, A = d(2, 70, 64).cuda(), d(2, 70, 1, 16).cuda(), -torch.rand(64, 16, generator=d.g).cuda()
    same = {"x": x, "dt": x, "Bm": bc, "Cm": bc, "z": x, "A": A}
    apart = {k: v.clone() for k, v in same.items()}
    assert torch.equal(la.forward_selective(**same), la.forward_selective(**apart))
    for u, v in zip(la.backward_selective(**same, dy=x), la.backward_selective(**apart, dy=x.clone())):
        assert u is v is None or torch.equal(u, v)
    assert torch.equal(la.forward_norm_residual(x, x)[0], la.forward_norm_residual(x, x.clone())[0])


def test_two_threads(la):
    """Calls from two host threads at once, each on a stream of its own."""
    import threading
    a, more, d = scan_inputs(BF16, (2, 300), 96, 16, 1, 13)
    args, dy = {**dev(a), **dev(more)}, d(2, 300, 96).cuda()
    want = la.backward_selective(**args, dy=dy)
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got = la.backward_selective(**args, dy=dy)
                    s.synchronize()
                    if not all(u is v is None or torch.equal(u, v) for u, v in zip(got, want)):
                        bad.append("other values")
        except Exception as e:  # noqa: BLE001 (reported by the assertion)
            bad.append(repr(e))

    ts = [threading.Thread(target=work) for _ in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad, bad


def test_block_prompt_then_tokens(la):
    """The operators together, as a block runs them: convolution, scan, gated
    norm, residual norm over a prompt with its states, then token by token; the
    outputs equal one pass over all the tokens."""
    B, L, more_tokens, E, N, W = 2, 130, 6, 128, 16, 4
    d = Draw(1, BF16)
    T = L + more_tokens
    x, dt = d(B, T, E), d(B, T, E)
    bc, gate, res = d(B, T, 2, 1, N), d(B, T, E), d(B, T, E)
    w, wb, A, D = d.f(E, W), d.f(E), -torch.rand(E, N, generator=d.g) - 0.1, d.f(E)
    dtb, wn, wr = d.f(E) - 3, d.f(2, 64), d.f(E)
    x, dt, bc, gate, res, w, wb, A, D, dtb, wn, wr = (
        t.cuda() for t in (x, dt, bc, gate, res, w, wb, A, D, dtb, wn, wr))

    def block(sl, conv_state=None, h0=None):
        c, cs = la.forward_conv(x[:, sl], w, wb, state=conv_state, return_state=True)
        y, h = la.forward_selective(c, dt[:, sl], A, bc[:, sl, 0], bc[:, sl, 1], D=D, dt_bias=dtb, h0=h0,
                                    return_state=True)
        n = la.forward_norm_gate(y.view(B, -1, 2, 64), gate[:, sl].contiguous(), wn, gate_first=True,
                                 heads_first=False)
        return la.forward_norm_residual(n, res[:, sl].contiguous(), wr) + (cs, h)

    whole = block(slice(0, T))
    # a prompt of B = 2 sequences as slices along the token axis
    xs = [t[:, :L].contiguous() for t in (x, dt, bc)]
    keep = (x, dt, bc)
    x, dt, bc = xs
    o, r, cs, h = block(slice(0, L))
    x, dt, bc = keep
    parts = [(o, r)]
    for t in range(L, T):
        c = la.decode_conv(x[:, t], w, cs, wb)
        y = la.decode_selective(c, dt[:, t], A, bc[:, t, 0], bc[:, t, 1], h, D=D, dt_bias=dtb)
        n = la.forward_norm_gate(y.view(B, 1, 2, 64), gate[:, t:t + 1].contiguous(), wn, gate_first=True,
                                 heads_first=False)
        parts.append(la.forward_norm_residual(n, res[:, t:t + 1].contiguous(), wr))
    assert torch.equal(cs, whole[2])
    # states: the same sums in another order of the parts
    assert torch.allclose(h, whole[3], rtol=0, atol=80 * T * 2.0 ** -24 * float(whole[3].abs().max()))
    for i in (0, 1):
        got = torch.cat([p[i] for p in parts], 1).float()
        # bf16 between the operators: two results that straddle a rounding border differ by a step
        # (2^-7 relative), in y and then in n
        size = whole[i].float().abs().amax(-1, keepdim=True)
        assert ((got - whole[i].float()).abs() <= 2.0 ** -5 * size).all()


def test_after_linear_attention(la):
    """The gated norm on la.forward's output, heads first as it returns it."""
    B, H, N, D = 2, 4, 200, 64
    d = Draw(8, BF16)
    q, k, v, gate, w = d(B, H, N, D), d(B, H, N, D), d(B, H, N, D), d(B, N, H * D), d.f(H, D)
    o = la.forward(q.cuda(), k.cuda(), v.cuda())
    n = la.forward_norm_gate(o, gate.cuda(), w.cuda())
    ref = osel.norm_gate(n64(o), gate.float().numpy(), w.numpy())
    close("norm gate after attention", n, ref, np.abs(ref), D / 8 + 32, BF16)


def test_streams_and_graphs(la):
    """Two captured graphs and an eager call of the same shapes on their own
    streams: workspaces are not shared, replays give the eager results."""
    B, L, E, N = 1, 600, 64, 16
    sets, want = [], []
    for seed in range(2):
        a, more, d = scan_inputs(BF16, (B, L), E, N, 1, 20 + seed)
        kw = {**dev(a), **dev(more)}
        dy, w = d(B, L, E).cuda(), d.f(E, 4).cuda()
        res = d.f(E).cuda()
        sets.append((kw, dy, w, res))

    def run(kw, dy, w, res):
        y, h = la.forward_selective(**kw, return_state=True)
        return [y, h, *la.backward_selective(**kw, dy=dy), *la.backward_conv(kw["x"], w, dy)[:2],
                *la.backward_norm_residual(y, dy, res)]

    want = [[t.clone() if t is not None else None for t in run(*s)] for s in sets]
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(*s)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = run(*sets[0])
    torch.cuda.synchronize()
    for got, ref in [(graphs[0][1], want[0]), (graphs[1][1], want[1]), (eager, want[0])]:
        for u, v in zip(got, ref):
            assert (u is None and v is None) or torch.equal(u, v)


def test_ragged_graph_replayed_with_other_lengths(la):
    """The lengths are read when a graph runs, not when it was captured."""
    B, L, E, N = 5, 900, 64, 16
    a, more, d = scan_inputs(BF16, (B, L), E, N, 1, 17)
    args = {**dev(a), **dev(more)}
    x, w = d(B, L, E).cuda(), d.f(E, 4).cuda()
    lens = torch.full((B,), L, dtype=torch.int32).cuda()
    y, h = torch.zeros(B, L, E, dtype=BF16).cuda(), torch.zeros(B, E, N).cuda()
    yc, sc = torch.zeros_like(y), torch.zeros(B, 3, E, dtype=BF16).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        la.forward_selective(**args, lens=lens, out=y, h=h)
        la.forward_conv(x, w, lens=lens, out=yc, state_out=sc)
    for new in ([L] * B, [0, 1, 33, 900, 500], [900, 0, 0, 0, 2]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        for t in (y, h, yc, sc):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = la.forward_selective(**args, lens=lens, out=torch.zeros_like(y), return_state=True)
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])
        want = la.forward_conv(x, w, lens=lens, out=torch.zeros_like(y), return_state=True)
        assert torch.equal(yc, want[0]) and torch.equal(sc, want[1])


def test_long_offsets(la):
    """Element offsets beyond 32 bits: the last sequence of a large batch."""
    B, L, E, W = 2, 1 << 20, 2048, 2
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.empty(B, L, E, dtype=BF16, device="cuda").normal_()
    w = torch.randn(E, W, device="cuda")
    y = la.forward_conv(x, w, silu=False)
    part = la.forward_conv(x[1:, -64:].contiguous(), w, silu=False)
    assert torch.equal(y[1, -63:], part[0, 1:])
    o, r = la.forward_norm_residual(x.view(-1, E))
    assert torch.equal(r[-3:], x.view(-1, E)[-3:])


@pytest.mark.parametrize("what", ["scan", "scan backward", "conv backward", "norm backward"])
def test_first_call_inside_a_capture(la, what):
    """A fresh process whose first call of all is captured, then replayed."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = f"""
import torch
import kernelized_sequence_mixing_gb300 as la
f = lambda *s: torch.randn(*s, device="cuda")
B, L, E, N = 1, 600, 64, 16
x, dt, A, Bm, Cm, dy, w = f(B, L, E), f(B, L, E), -torch.rand(E, N, device="cuda"), f(B, L, 1, N), f(B, L, 1, N), \
    f(B, L, E), f(E, 4)
call = {{"scan": lambda: la.forward_selective(x, dt, A, Bm, Cm),
        "scan backward": lambda: la.backward_selective(x, dt, A, Bm, Cm, dy)[0],
        "conv backward": lambda: la.backward_conv(x, w, dy)[0],
        "norm backward": lambda: la.backward_norm_residual(x, dy, w=A[:, 0].contiguous())[2]}}[{what!r}]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = call()
g.replay()
torch.cuda.synchronize()
assert torch.equal(got, call())
print("equal")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-1500:]


def plain_step(a, more, h):
    """One token in 64 bits on the GPU (many sequences)."""
    d = {k: v.double() for k, v in {**a, **more}.items()}
    E = d["x"].shape[1]
    rep = lambda m: m.repeat_interleave(E // m.shape[1], 1)  # noqa: E731
    step = torch.logaddexp(d["dt"] + d["dt_bias"], torch.zeros((), dtype=torch.float64, device="cuda"))
    new = torch.exp(step[..., None] * d["A"]) * h.double() + (step * d["x"])[..., None] * rep(d["Bm"])
    return ((new * rep(d["Cm"])).sum(-1) + d["D"] * d["x"]) * d["z"] * torch.sigmoid(d["z"]), new


def test_many_sequences(la):
    """More sequences than a grid has rows, for one token and for short prompts."""
    B, E, N = 140000, 8, 8
    a, more, d = scan_inputs(F32, (B,), E, N, 1, 4)
    a, more = dev(a), dev(more)
    h = torch.randn(B, E, N, device="cuda")
    hc = h.clone()
    y = la.decode_selective(**a, h=hc, **more)
    ry, rh = plain_step(a, more, h)
    assert float((hc - rh).abs().max()) < 400 * 2.0 ** -24 * float(rh.abs().max())
    assert float((y - ry).abs().max()) < 400 * 2.0 ** -24 * float(ry.abs().max()) + 400 * 2.0 ** -24 * 30
    seq = {k: (v[:, None] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in {**a, **more}.items()}
    y2, h2 = la.forward_selective(**seq, h0=h, return_state=True)
    assert float((h2 - rh).abs().max()) < 400 * 2.0 ** -24 * float(rh.abs().max())
    w, st = torch.randn(E, 4, device="cuda"), torch.randn(B, 3, E, device="cuda")
    full = (torch.cat((st, a["x"][:, None]), 1).double() * w.t().double()).sum(1)
    yc = la.decode_conv(a["x"], w, st, silu=False)
    assert float((yc - full).abs().max()) < 16 * 2.0 ** -24 * 60
    assert torch.equal(st[:, 2], a["x"])


@pytest.mark.parametrize("N", [8, 16, 64])
def test_long_sequence(la, N):
    """The largest number of parts, and its gradients."""
    B, L, E = 1, 9001, 16
    a, more, d = scan_inputs(F32, (B, L), E, N, 1, N)
    y, h = la.forward_selective(**dev(a), **dev(more), return_state=True)
    (ry, rh), (my, mh) = scan_ref(a, more, True)
    # a state forgets: with decays of at most exp(-0.05 x 0.003) its memory is under 7000 tokens
    close("scan long y", y, ry, my, 80 * 7000, F32)
    close("scan long state", h, rh, mh, 80 * 7000, F32)
    assert float((y.double() - torch.from_numpy(ry).cuda()).norm() / np.linalg.norm(ry)) < 2e-5
    dy = d(B, L, E)
    got = la.backward_selective(**dev(a), dy=dy.cuda(), **dev(more))
    ref = osel.scan_backward(**host(a), **host(more), dy=dy.numpy())
    for name, v in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias"), got):
        assert np.linalg.norm(n64(v) - ref[name]) <= 2e-5 * np.linalg.norm(ref[name]), name


def test_wide_batches_of_groups(la):
    """Many channel tiles and groups, with tails, against the parts alone: a
    group's channels give the same bits as that group on its own."""
    B, L, E, N, G = 2, 100, 1200, 16, 3
    a, more, d = scan_inputs(BF16, (B, L), E, N, G, 6)
    a, more, dy = dev(a), dev(more), d(B, L, E).cuda()
    y = la.forward_selective(**a, **more)
    got = la.backward_selective(**a, dy=dy, **more)
    for g in range(G):
        c = slice(g * E // G, (g + 1) * E // G)
        one = {k: (v[..., c].contiguous() if k in ("x", "dt", "D", "z", "dt_bias") else
                   v[c].contiguous() if k == "A" else v[:, :, g:g + 1].contiguous())
               for k, v in {**a, **more}.items()}
        assert torch.equal(la.forward_selective(**one), y[..., c])
        part = la.backward_selective(**one, dy=dy[..., c].contiguous())
        for i, v in enumerate(part):
            if v is None:
                continue
            whole = got[i][:, :, g:g + 1] if i in (3, 4) else got[i][c] if i in (2, 5, 7) else got[i][..., c]
            assert torch.equal(v, whole), i
