"""Retention and beam search without a GPU: refusals of the C entry points and
of the binding before any CUDA call, and the fp64 oracle against closed forms
and differences."""
import ctypes

import numpy as np
import pytest
import torch

import kernelized_sequence_mixing_gb300 as la
from oracle import retention as ort

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32C, BF16C = 0, 1
P0, STEP = 0x10000000, 0x10000000  # fake device addresses, never touched


@pytest.fixture(scope="module")
def lib():
    from kernelized_sequence_mixing_gb300 import build
    build.build()
    return la.load_library()


class Call:
    """A C entry point with good arguments by name; keywords change some."""

    def __init__(self, fn, names, more):
        self.fn, self.names = fn, names.split()
        self.good = {**{n: P0 + i * STEP for i, n in enumerate(self.names)}, **more}

    def __call__(self, **kw):
        a = {**self.good, **kw}
        return self.fn(*(a[n] for n in self.good), None)


SIZES = {"B": 2, "L": 5, "H": 4, "Hk": 2, "D": 64, "Dv": 32, "strides": None, "gamma": None, "scale": 1.0, "dtype": BF16C}


def floats(*v):
    return (ctypes.c_float * len(v))(*v)


def strides(q=(1280, 256, 64), k=(640, 128, 64), v=(320, 64, 32), o=(640, 128, 32)):
    return (ctypes.c_longlong * 12)(*q, *k, *v, *o)


def common_refusals(c, dims=True):
    assert c(D=60) == UNSUPPORTED and c(Dv=264) == UNSUPPORTED and c(D=0) == INVALID
    assert c(H=3) == INVALID and c(Hk=0) == INVALID and c(Hk=8) == INVALID
    assert c(H=514, Hk=2) == UNSUPPORTED
    assert c(B=-1) == INVALID and c(dtype=7) == INVALID
    for bad in (0.0, float("inf"), float("nan")):
        assert c(scale=bad) == INVALID
    for bad in (-0.1, 1.5, float("nan")):
        assert c(gamma=floats(1, 1, 1, bad)) == INVALID
    none = {n: None for n in c.names}
    assert c(**none, B=0) == OK and c(**none, H=0, Hk=0) == OK


def test_scales_beyond_the_range(lib):
    """The backward pass divides by the scale: both calls refuse one whose inverse
    or whose products would leave fp32."""
    for name, names in (("la_forward_retention", "q k v S0 lens o S"),
                        ("la_backward_retention", "q k v dO S0 dS lens dq dk dv dS0")):
        c = Call(getattr(lib, name), names, SIZES)
        for bad in (1e-39, 2.0 ** -65, -2.0 ** -70, 2.0 ** 65, -3e38):
            assert c(scale=bad) == INVALID
        assert c(scale=2.0 ** -64, B=0) == OK and c(scale=-2.0 ** 64, B=0) == OK


def test_forward_refusals(lib):
    c = Call(lib.la_forward_retention, "q k v S0 lens o S", SIZES)
    for name in ("q", "k", "v", "o"):
        assert c(**{name: None}) == INVALID, name
    for name in ("q", "k", "v", "S0", "o", "S"):
        assert c(**{name: c.good[name] + 8}) == INVALID, name
    common_refusals(c)
    assert c(B=1 << 16, L=1 << 15) == UNSUPPORTED
    assert c(B=1 << 25, H=4) == UNSUPPORTED
    assert c(S=c.good["S0"]) == INVALID            # in place
    assert c(o=c.good["q"]) == INVALID and c(S=c.good["lens"]) == INVALID and c(o=c.good["lens"]) == INVALID
    assert c(lens=c.good["lens"] + 2) == INVALID
    # strides: not multiples of 8, rows over one another, negative, a zero
    for bad in (strides(q=(1280, 252, 64)), strides(k=(640, 128, 32)), strides(v=(320, -64, 32)),
                strides(o=(640, 128, 0)), strides(o=(512, 128, 32)), strides(q=(0, 256, 64))):
        assert c(strides=bad) == INVALID
    # a stride that makes q reach into o
    assert c(strides=strides(q=(5 * STEP // 2, 256, 64))) == INVALID
    none = {n: None for n in c.names}
    assert c(**none, L=0) == OK                    # no tokens, no state wanted


def test_backward_refusals(lib):
    c = Call(lib.la_backward_retention, "q k v dO S0 dS lens dq dk dv dS0", SIZES)
    for name in ("q", "k", "v", "dO", "dq", "dk", "dv", "S0"):
        assert c(**{name: None}) == INVALID, name
    common_refusals(c)
    assert c(dS0=c.good["dS"]) == INVALID and c(dq=c.good["q"]) == INVALID and c(dk=c.good["dv"]) == INVALID
    assert c(dv=c.good["lens"]) == INVALID
    none = {n: None for n in c.names}
    assert c(**none, L=0) == OK


def test_decode_refusals(lib):
    sizes = {"B": 3, "pool": 4, "H": 4, "Hk": 2, "D": 64, "Dv": 32, "ldq": 0, "ldk": 0, "ldv": 0, "gamma": None,
             "scale": 1.0, "dtype": BF16C}
    c = Call(lib.la_decode_retention, "q k v S slots o", sizes)
    for name in ("q", "k", "v", "S", "o"):
        assert c(**{name: None}) == INVALID, name
        assert c(**{name: c.good[name] + 4}) == INVALID, name
    common_refusals(c)
    assert c(slots=None, pool=2) == INVALID        # fewer states than sequences
    assert c(pool=-1) == INVALID and c(slots=c.good["slots"] + 1) == INVALID
    assert c(o=c.good["S"]) == INVALID and c(S=c.good["slots"]) == INVALID
    assert c(ldq=248) == INVALID and c(ldk=132) == INVALID and c(ldv=-64) == INVALID
    assert c(pool=0) == OK                         # every slot is outside
    assert c(pool=1 << 30, H=4) == UNSUPPORTED


def test_select_refusals(lib):
    sizes = {"B": 2, "K": 4, "V": 100, "n": 8, "ld": 0, "eos": 2, "dtype": BF16C}
    c = Call(lib.la_select_beams, "logits scores finished out_scores parents tokens", sizes)
    for name in ("logits", "scores", "out_scores", "parents", "tokens"):
        assert c(**{name: None}) == INVALID, name
        assert c(**{name: c.good[name] + 1}) == INVALID, name
    assert c(K=0) == INVALID and c(V=0) == INVALID and c(n=0) == INVALID and c(n=401) == INVALID
    assert c(K=33) == UNSUPPORTED and c(n=65) == UNSUPPORTED and c(V=(1 << 30) + 1) == UNSUPPORTED
    assert c(B=1 << 25) == UNSUPPORTED and c(ld=99) == INVALID and c(dtype=3) == INVALID
    assert c(eos=100) == INVALID and c(eos=-1) == INVALID
    assert c(parents=c.good["tokens"]) == INVALID and c(out_scores=c.good["scores"]) == INVALID
    assert c(**{n: None for n in c.names}, B=0) == OK


def test_reorder_refusals(lib):
    def call(ptrs, sizes, parents=P0, B=2, K=4):
        n = len(sizes)
        p = (ctypes.c_void_p * n)(*ptrs) if ptrs is not None else None
        return lib.la_reorder_states(p, (ctypes.c_longlong * n)(*sizes), n, parents, B, K, None)

    a, b = P0 + STEP, P0 + 2 * STEP
    assert call([a, b], [64, 64], parents=None) == INVALID
    assert call([a, b], [64, 64], parents=P0 + 1) == INVALID
    assert call([a, None], [64, 64]) == INVALID and call([a, b], [64, -1]) == INVALID
    assert call([a, a + 64], [64, 64]) == INVALID          # over one another
    assert call([a, P0 - 64], [64, 64]) == INVALID         # over the parents
    assert call(None, [64]) == INVALID
    assert call([a], [64], K=0) == INVALID and call([a], [64], K=33) == UNSUPPORTED
    assert call([a], [64], B=0) == OK and call([], [], parents=None) == OK


# --- the binding, on host tensors: every refusal comes before the device check ---

def qkv(B=2, L=3, H=4, Hk=2, D=64, Dv=32, dtype=torch.float32):
    return torch.zeros(B, L, H, D, dtype=dtype), torch.zeros(B, L, Hk, D, dtype=dtype), torch.zeros(B, L, Hk, Dv, dtype=dtype)


def test_binding_refusals():
    q, k, v = qkv()
    with pytest.raises(ValueError, match="CUDA"):
        la.forward_retention(q, k, v)
    with pytest.raises(ValueError, match="divide"):
        la.forward_retention(q[:, :, :3], k, v)
    with pytest.raises(ValueError, match="shape"):
        la.forward_retention(q, k[..., :32], v)
    with pytest.raises(TypeError):
        la.forward_retention(q, k.bfloat16(), v)
    with pytest.raises(TypeError):
        la.forward_retention(q.half(), k.half(), v.half())
    with pytest.raises(ValueError, match="contiguous"):
        la.forward_retention(q.transpose(2, 3).contiguous().transpose(2, 3), k, v)
    with pytest.raises(ValueError, match="apart"):
        la.forward_retention(q, k[:, :, :1].expand(2, 3, 2, 64), v)
    with pytest.raises(ValueError, match="apart"):
        la.forward_retention(torch.zeros(2, 3, 4, 68)[..., :64], k, v)
    for bad in (dict(S0=torch.zeros(2, 4, 64, 31)), dict(S=torch.zeros(2, 4, 32, 64)), dict(out=torch.zeros(2, 3, 4, 64)),
                dict(lens=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            la.forward_retention(q, k, v, **bad)
    with pytest.raises(TypeError):
        la.forward_retention(q, k, v, lens=torch.zeros(2))
    with pytest.raises(ValueError, match="shape"):
        la.backward_retention(q, k, v, torch.zeros(2, 3, 4, 64))
    with pytest.raises(ValueError, match="shape"):
        la.decode_retention(q[:, 0], k[:, 0], v[:, 0], torch.zeros(3, 4, 64, 32))
    with pytest.raises(TypeError):
        la.decode_retention(q[:, 0], k[:, 0], v[:, 0], torch.zeros(3, 4, 64, 32), slots=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="between 1 and"):
        la.select_beams(torch.zeros(2, 2, 3), torch.zeros(2, 2), n=7)
    with pytest.raises(ValueError, match="eos"):
        la.select_beams(torch.zeros(2, 2, 3), torch.zeros(2, 2), finished=torch.zeros(2, 2, dtype=torch.bool))
    with pytest.raises(ValueError, match="evenly"):
        la.select_beams(torch.zeros(2, 3, 2).transpose(1, 2), torch.zeros(2, 2))
    with pytest.raises(TypeError):
        la.select_beams(torch.zeros(2, 2, 3), torch.zeros(2, 2, dtype=torch.float64))
    parents = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be"):
        la.reorder_states([torch.zeros(2, 3, 8)], parents)
    with pytest.raises(ValueError, match="contiguous"):
        la.reorder_states(torch.zeros(2, 4, 8)[..., :4], parents)
    with pytest.raises(TypeError):
        la.reorder_states([torch.zeros(2, 4, 8)], parents.long())


# --- the oracle ---

def draw(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def problem(B=2, L=7, H=4, Hk=2, D=3, Dv=5):
    return (draw(1, B, L, H, D), draw(2, B, L, Hk, D), draw(3, B, L, Hk, Dv), draw(4, B, H, D, Dv),
            np.array([1.0, 0.9, 0.5, 0.0])[:H])


def test_oracle_quadratic_form():
    q, k, v, S0, g = problem()
    lens = [7, 4]
    o, S = ort.forward(q, k, v, g, 0.7, S0, lens)
    for b in range(2):
        for h in range(4):
            n = lens[b]
            i = np.arange(n)
            far = i[:, None] - i
            w = np.where(far >= 0, g[h] ** np.maximum(far, 0), 0) * (q[b, :n, h] @ k[b, :n, h // 2].T)
            ref = 0.7 * (w @ v[b, :n, h // 2] + (g[h] ** (i + 1))[:, None] * (q[b, :n, h] @ S0[b, h]))
            np.testing.assert_allclose(o[b, :n, h], ref, rtol=1e-12, atol=1e-12)
            end = (k[b, :n, h // 2] * (g[h] ** (n - 1 - i))[:, None]).T @ v[b, :n, h // 2] + g[h] ** n * S0[b, h]
            np.testing.assert_allclose(S[b, h], end, rtol=1e-12, atol=1e-12)
    assert not o[1, 4:].any()


def test_oracle_gradients_are_differences():
    q, k, v, S0, g = problem(L=5)
    do, dS, lens = draw(5, 2, 5, 4, 5), draw(6, *S0.shape), [5, 3]
    grads = ort.backward(q, k, v, do, g, 0.7, S0, dS, lens)

    def loss():
        o, S = ort.forward(q, k, v, g, 0.7, S0, lens)
        return (o * do)[0].sum() + (o * do)[1, :3].sum() + (S * dS).sum()

    rng = np.random.default_rng(7)
    for x, gx in zip((q, k, v, S0), grads):
        way = rng.standard_normal(x.shape)
        x += 1e-4 * way
        up = loss()
        x -= 2e-4 * way
        down = loss()
        x += 1e-4 * way
        # the loss is a polynomial: the central difference is off by third-order terms of 1e-8
        assert abs((up - down) / 2e-4 - (gx * way).sum()) < 1e-5
    assert not grads[0][1, 3:].any() and not grads[1][1, 3:].any() and not grads[2][1, 3:].any()


def test_oracle_selection():
    x = np.log(np.array([[[0.5, 0.25, 0.25], [0.8, 0.1, 0.1]]]))
    s, p, t = ort.select(x, np.log(np.array([[0.5, 0.25]])), 4)
    np.testing.assert_allclose(np.exp(s), [[0.25, 0.2, 0.125, 0.125]])
    assert p.tolist() == [[0, 1, 0, 0]] and t.tolist() == [[0, 0, 1, 2]]
    s, p, t = ort.select(x, np.log(np.array([[0.5, 0.25]])), 4, np.array([[False, True]]), 1)
    np.testing.assert_allclose(np.exp(s), [[0.25, 0.25, 0.125, 0.125]])
    assert sorted(zip(p[0, :2], t[0, :2])) == [(0, 0), (1, 1)] and p[0, 2:].tolist() == [0, 0] and t[0, 2:].tolist() == [1, 2]
