"""The selective scan, its convolution and the norms without a GPU: the C
entry points refuse bad arguments before any CUDA call, the binding refuses bad
tensors before it loads the library, and the fp64 oracle agrees with
differences and with closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import kernelized_sequence_mixing_gb300 as la
from oracle import selective as osel

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32C, BF16C = 0, 1
P0, STEP = 0x10000000, 0x10000000  # fake device addresses, never touched


@pytest.fixture(scope="module")
def lib():
    from kernelized_sequence_mixing_gb300 import build
    build.build()
    return la.load_library()


def ptrs(names):
    return {n: P0 + i * STEP for i, n in enumerate(names.split())}


class Call:
    """A C entry point with good arguments by name; keywords change some."""

    def __init__(self, fn, names, sizes):
        self.fn, self.names = fn, names.split()
        self.good = {**ptrs(names), **sizes}

    def __call__(self, **kw):
        a = {**self.good, **kw}
        return self.fn(*(a[n] for n in list(self.good)), None)


SCAN = "x dt A Bm Cm D z dt_bias"
LDS = {"ldx": 0, "lddt": 0, "ldz": 0, "ldb": 0, "ldc": 0, "softplus": 1, "dtype": BF16C}


def test_forward_selective_refusals(lib):
    c = Call(lib.la_forward_selective, SCAN + " h0 lens y hN",
             {"B": 2, "L": 5, "E": 64, "N": 16, "G": 2, **LDS})
    for name in ("x", "dt", "A", "Bm", "Cm", "y"):
        assert c(**{name: None}) == INVALID, name
        assert c(**{name: c.good[name] + 8}) == INVALID, name
    assert c(hN=c.good["h0"]) == INVALID           # in place
    assert c(y=c.good["z"] + 64) == INVALID
    assert c(hN=c.good["lens"]) == INVALID
    assert c(lens=c.good["lens"] + 2) == INVALID
    assert c(B=-1) == INVALID and c(N=0) == INVALID and c(G=0) == INVALID and c(dtype=5) == INVALID
    assert c(G=3) == INVALID                       # 64 channels in 3 groups
    assert c(G=16) == UNSUPPORTED                  # 4 channels a group
    assert c(E=60) == UNSUPPORTED and c(N=12) == UNSUPPORTED and c(E=65544) == UNSUPPORTED
    assert c(B=1 << 16, L=1 << 15) == UNSUPPORTED
    assert c(B=1 << 26, L=1) == UNSUPPORTED        # 2^32 channels
    for ld, w in (("ldx", 64), ("lddt", 64), ("ldz", 64), ("ldb", 32), ("ldc", 32)):
        assert c(**{ld: w - 8}) == INVALID and c(**{ld: w + 4}) == INVALID and c(**{ld: -w}) == INVALID
    # a stride makes the input reach into y
    assert c(ldx=8 * STEP) == INVALID
    none = {n: None for n in c.names}
    assert c(**none, B=0) == OK and c(**none, E=0) == OK


def test_decode_selective_refusals(lib):
    c = Call(lib.la_decode_selective, SCAN + " h y", {"B": 2, "E": 64, "N": 16, "G": 1, **LDS})
    for name in ("x", "dt", "A", "Bm", "Cm", "h", "y"):
        assert c(**{name: None}) == INVALID, name
    assert c(y=c.good["x"]) == INVALID and c(h=c.good["y"]) == INVALID
    assert c(ldx=72 + 4) == INVALID
    assert c(N=128) == UNSUPPORTED
    assert c(**{n: None for n in c.names}, B=0) == OK


def test_backward_selective_refusals(lib):
    c = Call(lib.la_backward_selective, SCAN + " h0 dy dhN dx ddt dA dBm dCm dD dz ddt_bias dh0",
             {"B": 2, "L": 5, "E": 64, "N": 16, "G": 1, **LDS})
    for name in ("x", "dt", "A", "Bm", "Cm", "dy", "dx", "ddt", "dA", "dBm", "dCm"):
        assert c(**{name: None}) == INVALID, name
    # gradients of inputs that are not there, z without dz
    assert c(D=None) == INVALID and c(dt_bias=None) == INVALID and c(h0=None) == INVALID
    assert c(z=None) == INVALID and c(dz=None) == INVALID
    assert c(dx=c.good["dy"]) == INVALID and c(dA=c.good["ddt_bias"]) == INVALID
    assert c(dh0=c.good["dhN"]) == INVALID         # in place
    assert c(E=36) == UNSUPPORTED
    assert c(**{n: None for n in c.names}, E=0) == OK


def test_conv_refusals(lib):
    sizes = {"B": 2, "L": 5, "E": 64, "W": 4, "ldx": 0, "silu": 1, "dtype": F32C}
    c = Call(lib.la_forward_conv, "x w bias state lens y state_out", sizes)
    for name in ("x", "w", "y"):
        assert c(**{name: None}) == INVALID, name
    assert c(W=0) == INVALID and c(W=1) == UNSUPPORTED and c(W=5) == UNSUPPORTED
    assert c(E=12) == UNSUPPORTED and c(y=c.good["x"]) == INVALID
    assert c(state_out=c.good["state"]) == INVALID and c(lens=c.good["lens"] + 1) == INVALID
    assert c(lens=c.good["y"] + 4) == INVALID
    assert c(ldx=56) == INVALID and c(ldx=68) == INVALID
    none = {n: None for n in c.names}
    assert c(**none, B=0) == OK
    assert c(L=0, x=None, y=None, state_out=None) == OK
    b = Call(lib.la_backward_conv, "x w bias state dy dx dw dbias dstate", sizes)
    for name in ("x", "w", "dy", "dx", "dw", "bias", "state"):
        assert b(**{name: None}) == INVALID, name
    assert b(dx=b.good["dy"]) == INVALID and b(dstate=b.good["state"]) == INVALID
    del sizes["L"]
    s = Call(lib.la_decode_conv, "x w bias state y", sizes)
    for name in ("x", "w", "state", "y"):
        assert s(**{name: None}) == INVALID, name
    assert s(y=s.good["state"] + 16) == INVALID
    assert s(**{n: None for n in s.names}, B=0) == OK


def test_norm_refusals(lib):
    sizes = {"B": 2, "H": 3, "L": 5, "D": 64, "hf": 1, "gf": 0, "eps": 1e-5, "dtype": BF16C}
    c = Call(lib.la_forward_norm_gate, "y gate w out", sizes)
    b = Call(lib.la_backward_norm_gate, "y gate w dout dy dgate dw", sizes)
    for call, need in ((c, "y gate out"), (b, "y gate dout dy dgate")):
        for name in need.split():
            assert call(**{name: None}) == INVALID, name
        assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
        assert call(D=0) == INVALID and call(H=-1) == INVALID and call(dtype=2) == INVALID
        assert call(D=68) == UNSUPPORTED and call(D=8200) == UNSUPPORTED
        assert call(H=1025) == UNSUPPORTED and call(B=1 << 20, L=1 << 10) == UNSUPPORTED
    assert c(out=c.good["gate"]) == INVALID and b(dy=b.good["dout"]) == INVALID
    assert b(w=None) == INVALID                    # dw without w
    assert c(**{n: None for n in c.names}, L=0) == OK
    sizes = {"rows": 9, "E": 64, "scale": 0.5, "eps": 1e-5, "dtype": BF16C}
    c = Call(lib.la_forward_norm_residual, "x residual w o r", sizes)
    b = Call(lib.la_backward_norm_residual, "r w dout dr dresidual dx dw", sizes)
    for call, need in ((c, "x o r"), (b, "r dout dresidual")):
        for name in need.split():
            assert call(**{name: None}) == INVALID, name
        assert call(scale=float("inf")) == INVALID and call(eps=-1.0) == INVALID
        assert call(rows=-1) == INVALID and call(E=4) == UNSUPPORTED and call(E=8200) == UNSUPPORTED
    assert c(r=c.good["residual"]) == INVALID and c(o=c.good["r"]) == INVALID
    assert b(dx=None) == INVALID                   # needed where scale is not 1
    assert c(**{n: None for n in c.names}, rows=0) == OK


# ------------------------------------------------------------------ binding

class Reached(Exception):
    pass


@pytest.fixture
def no_library(monkeypatch):
    def stop():
        raise Reached

    monkeypatch.setattr(la, "load_library", stop)
    monkeypatch.setattr(la, "_DEVICE_TYPES", ("cuda", "meta"))


BF, F32 = torch.bfloat16, torch.float32
B, L, E, N, G = 2, 6, 64, 16, 2


def T(*shape, dtype=BF, device="meta"):
    return torch.empty(shape, dtype=dtype, device=device)


def F(*shape):
    return T(*shape, dtype=F32)


def scan_args(lead=(B, L)):
    return {"x": T(*lead, E), "dt": T(*lead, E), "A": F(E, N), "Bm": T(*lead, G, N), "Cm": T(*lead, G, N),
            "D": F(E), "z": T(*lead, E), "dt_bias": F(E)}


def passes(fn, **kw):
    with pytest.raises(Reached):
        fn(**kw)


def fails(exc, fn, **kw):
    with pytest.raises(exc):
        fn(**kw)


def test_selective_binding(no_library):
    a = scan_args()
    more = {"h0": F(B, E, N), "lens": T(B, dtype=torch.int32), "out": T(B, L, E), "h": F(B, E, N)}
    passes(la.forward_selective, **a, **more)
    xz = T(B, L, 2 * E)
    passes(la.forward_selective, **{**a, "x": xz[..., :E], "z": xz[..., E:]})
    passes(la.forward_selective, **{**a, "Bm": T(B, L, 2, G, N)[:, :, 1]})
    passes(la.backward_selective, **a, dy=T(B, L, E), h0=F(B, E, N), dh=F(B, E, N))
    step = scan_args((B,))
    passes(la.decode_selective, **step, h=F(B, E, N))
    passes(la.decode_selective, **{**step, "x": xz[:, 0, :E]}, h=F(B, E, N))
    for fn, args in ((la.forward_selective, a), (la.backward_selective, {**a, "dy": T(B, L, E)}),
                     (la.decode_selective, {**step, "h": F(B, E, N)})):
        lead = args["x"].shape[:-1]
        fails(ValueError, fn, **{**args, "dt": T(*lead, E + 8)})
        fails(TypeError, fn, **{**args, "z": F(*lead, E)})
        fails(TypeError, fn, **{**args, "A": T(E, N)})
        fails(ValueError, fn, **{**args, "A": F(N, E).t()})
        fails(ValueError, fn, **{**args, "Cm": T(*lead, G, N + 8)})
        fails(ValueError, fn, **{**args, "Bm": T(*lead, N)})
        fails(ValueError, fn, **{**args, "D": F(E, 1)})
        fails(TypeError, fn, **{**args, "x": T(*lead, E, dtype=torch.float16)})
        fails(ValueError, fn, **{**args, "x": T(*lead, E, device="cpu")})
        fails(ValueError, fn, **{**args, "x": T(*lead, 2 * E)[..., ::2]})   # gaps in a row
        fails(ValueError, fn, **{**args, "x": T(*lead, E + 4)[..., :E]})    # stride not of 8
        fails(ValueError, fn, **{**args, "x": T(1, E).expand(*lead, E) if len(lead) == 1
                                 else T(1, 1, E).expand(*lead, E)})         # broadcast
    fails(ValueError, la.forward_selective, **{**a, "x": T(B, L + 2, E)[:, :L]})  # batch stride
    fails(TypeError, la.forward_selective, **a, lens=T(B, dtype=torch.int64))
    fails(ValueError, la.forward_selective, **a, h0=F(B, N, E))
    fails(ValueError, la.forward_selective, **a, out=T(B, E, L).transpose(1, 2))
    fails(ValueError, la.backward_selective, **a, dy=T(B, L, 2 * E)[..., :E])
    fails(TypeError, la.decode_selective, **step, h=T(B, E, N))


def test_conv_binding(no_library):
    x, w = T(B, L, E), F(E, 4)
    passes(la.forward_conv, x=x, w=w, bias=F(E), state=T(B, 3, E), state_out=T(B, 3, E))
    passes(la.backward_conv, x=T(B, L, 2 * E)[..., E:], w=w, dy=x)
    passes(la.decode_conv, x=T(B, E), w=w, state=T(B, 3, E))
    fails(ValueError, la.forward_conv, x=x, w=F(4, E))
    fails(TypeError, la.forward_conv, x=x, w=T(E, 4))
    fails(ValueError, la.forward_conv, x=x, w=w, state=T(B, 4, E))
    fails(TypeError, la.forward_conv, x=x, w=w, state=F(B, 3, E))
    fails(ValueError, la.forward_conv, x=x[0], w=w)
    fails(ValueError, la.backward_conv, x=x, w=w, dy=T(B, L + 1, E))
    fails(ValueError, la.decode_conv, x=x, w=w, state=T(B, 3, E))
    fails(ValueError, la.decode_conv, x=T(B, E), w=w, state=T(B, 2, E))


def test_norm_binding(no_library):
    y, g = T(B, 3, L, 64), T(B, L, 192)
    passes(la.forward_norm_gate, y=y, gate=g, w=F(3, 64))
    passes(la.forward_norm_gate, y=T(B, L, 3, 64), gate=g, heads_first=False, out=T(B, L, 192))
    passes(la.backward_norm_gate, y=y, gate=g, do=g, w=F(3, 64))
    fails(ValueError, la.forward_norm_gate, y=T(B, L, 3, 64), gate=g)      # tokens first
    fails(ValueError, la.forward_norm_gate, y=y, gate=g, w=F(192))
    fails(TypeError, la.forward_norm_gate, y=y, gate=F(B, L, 192))
    fails(ValueError, la.backward_norm_gate, y=y, gate=g, do=y)
    fails(ValueError, la.forward_norm_gate, y=y.transpose(2, 3), gate=g)
    x = T(7, 64)
    passes(la.forward_norm_residual, x=x, residual=x, w=F(64))
    passes(la.backward_norm_residual, r=x, do=x, dr=x, w=F(64), scale=0.5)
    fails(ValueError, la.forward_norm_residual, x=x, residual=T(8, 64))
    fails(TypeError, la.forward_norm_residual, x=x, w=T(64))
    fails(ValueError, la.backward_norm_residual, r=x, do=T(7, 128)[:, :64])


# ------------------------------------------------------------------- oracle

def draws(seed):
    r = np.random.default_rng(seed)
    b, l, e, n, g = 2, 5, 6, 3, 2
    p = {"x": r.normal(size=(b, l, e)), "dt": r.normal(size=(b, l, e)), "A": -r.random((e, n)),
         "Bm": r.normal(size=(b, l, g, n)), "Cm": r.normal(size=(b, l, g, n)), "D": r.normal(size=e),
         "z": r.normal(size=(b, l, e)), "dt_bias": r.normal(size=e), "h0": r.normal(size=(b, e, n))}
    return p, r.normal(size=(b, l, e)), r.normal(size=(b, e, n)), r


def slope(f, p, v):
    s = 1e-5
    return (f({k: p[k] + s * v[k] for k in p}) - f({k: p[k] - s * v[k] for k in p})) / (2 * s)


def check_slopes(f, p, grads, r):
    """Directional derivatives, one input at a time."""
    for k in p:
        v = {q: np.zeros_like(p[q]) for q in p}
        v[k] = r.normal(size=p[k].shape)
        want = slope(f, p, v)
        assert abs(want - (grads[k] * v[k]).sum()) < 1e-7 * (1 + abs(want)), k


@pytest.mark.parametrize("sp", [True, False])
def test_oracle_scan_gradients(sp):
    p, dy, dh, r = draws(1)

    def loss(q):
        y, h = osel.scan(**q, softplus_dt=sp)
        return (y * dy).sum() + (h * dh).sum()

    g = osel.scan_backward(**p, dy=dy, dh=dh, softplus_dt=sp)
    names = {"x": "dx", "dt": "ddt", "A": "dA", "Bm": "dB", "Cm": "dC", "D": "dD", "z": "dz",
             "dt_bias": "ddt_bias", "h0": "dh0"}
    check_slopes(loss, p, {k: g[n] for k, n in names.items()}, r)


def test_oracle_scan_closed_form():
    """Constant step and decay: h_t is a geometric sum."""
    L_, a, step = 7, -0.5, 0.3
    one = np.ones((1, L_, 1))
    y, h = osel.scan(one, step * one, np.full((1, 1), a), one[..., None], one[..., None],
                     softplus_dt=False)
    q = np.exp(step * a)
    want = step * (1 - q ** np.arange(1, L_ + 1)) / (1 - q)
    assert np.allclose(y[0, :, 0], want, rtol=1e-14) and np.isclose(h[0, 0, 0], want[-1], rtol=1e-14)


def test_oracle_conv_gradients_and_taps():
    r = np.random.default_rng(2)
    p = {"x": r.normal(size=(2, 5, 3)), "w": r.normal(size=(3, 4)), "bias": r.normal(size=3),
         "state": r.normal(size=(2, 3, 3))}
    dy = r.normal(size=(2, 5, 3))
    for act in (True, False):
        g = osel.conv_backward(**p, dy=dy, silu_act=act)
        check_slopes(lambda q: (osel.conv(**q, silu_act=act)[0] * dy).sum(), p,  # noqa: B023
                     {"x": g["dx"], "w": g["dw"], "bias": g["dbias"], "state": g["dstate"]}, r)
    # w = the last tap alone is the identity, the first a shift by W - 1
    w = np.zeros((3, 4))
    w[:, 3] = 1
    assert np.array_equal(osel.conv(p["x"], w, silu_act=False)[0], p["x"])
    y, st = osel.conv(p["x"], w[:, ::-1], silu_act=False)
    assert np.array_equal(y[:, 3:], p["x"][:, :-3]) and (y[:, :3] == 0).all()
    assert np.array_equal(st, p["x"][:, -3:])


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("heads", [True, False])
def test_oracle_norm_gradients(first, heads):
    r = np.random.default_rng(3)
    p = {"y": r.normal(size=(2, 3, 4, 8) if heads else (2, 4, 3, 8)), "gate": r.normal(size=(2, 4, 24)),
         "w": r.normal(size=(3, 8))}
    do = r.normal(size=(2, 4, 24))
    kw = {"gate_first": first, "heads_first": heads, "eps": 0.1}
    g = osel.norm_gate_backward(**p, do=do, **kw)
    check_slopes(lambda q: (osel.norm_gate(**q, **kw) * do).sum(), p,
                 {"y": g["dy"], "gate": g["dgate"], "w": g["dw"]}, r)


def test_oracle_residual_gradients():
    r = np.random.default_rng(4)
    p = {"x": r.normal(size=(4, 8)), "residual": r.normal(size=(4, 8)), "w": r.normal(size=8)}
    do, dr = r.normal(size=(4, 8)), r.normal(size=(4, 8))

    def loss(q):
        o, s = osel.norm_residual(**q, scale=0.5, eps=0.1)
        return (o * do).sum() + (s * dr).sum()

    g = osel.norm_residual_backward(osel.norm_residual(**p, scale=0.5)[1], do, p["w"], dr, 0.5, 0.1)
    check_slopes(loss, p, {"x": g["dx"], "residual": g["dresidual"], "w": g["dw"]}, r)


def test_magnitudes_bound_the_values():
    p, dy, dh, _ = draws(5)
    for a, b in zip(osel.scan(**p), osel.scan(**p, mag=True)):
        assert (np.abs(a) <= b * (1 + 1e-12)).all()
    g, m = (osel.scan_backward(**p, dy=dy, dh=dh, mag=k) for k in (False, True))
    for k in g:
        assert (np.abs(g[k]) <= m[k] * (1 + 1e-12)).all(), k


def test_ctypes_signatures_match_the_header():
    """Every entry point's argument count, pointers and sizes in order."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "linattn.h")).read(), flags=re.S)
    lib = la.load_library()
    kinds = {ctypes.c_void_p: "P", ctypes.c_int: "I", ctypes.c_longlong: "LL", ctypes.c_float: "F"}
    seen = 0
    for name, args in re.findall(r"LA_API\s+la_status_t\s+(la_\w+)\s*\((.*?)\);", src, flags=re.S):
        if "selective" not in name and "conv" not in name and "norm" not in name:
            continue
        want = []
        for arg in args.split(","):
            arg = " ".join(arg.split())
            want.append("P" if "*" in arg else "LL" if "long long" in arg else "F" if "float" in arg else "I")
        assert [kinds[t] for t in getattr(lib, name).argtypes] == want, name
        seen += 1
    assert seen == 10
