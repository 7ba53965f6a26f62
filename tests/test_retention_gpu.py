"""GPU parity of retention and of beam search over its states against the fp64
oracle.

Tolerances, element by element, with mag the element's sums over absolute
values (from the oracle):

  half a step of the output's type, relative to the value, plus
  K 2^-24 mag, K = 2 L + 2 D + 64 (group sums: + H / Hk): the fp32 roundings on
  the longest path -- one multiplication by a power of the decay and one sum per
  chunk at most and two per token, the D products of a weight, and a power
  2^(e log2 g) that is off by e |log2 g| 2^-24 with |log2 g| <= 1 here (e <= L);
  bf16 outputs of the tensor-core kernel also 2^-8 mag (each product meets one
  factor that was rounded to bf16: within a chunk its weight, further back the
  decayed row that built the state) + 2^-15 mag (states as sums of two bf16
  values, 2^-16, and the second order).

States that are returned are fp32 (decayed rows as three bf16 values, 2^-24).
"""
import numpy as np
import pytest
import torch

from helpers import record
from oracle import retention as ort

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DT = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
sid = lambda s: "x".join(map(str, s))  # noqa: E731


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


def close(name, got, ref, mag, K, dtype, products=False):
    got = n64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), name
    if not got.size:
        return
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + K * 2.0 ** -24 * mag + 1e-37
    if products and dtype == BF16:
        tol = tol + (2.0 ** -8 + 2.0 ** -15) * mag
    worst = float((np.abs(got - ref) / tol).max())
    record(f"retention {name} {str(dtype)[6:]} (share of its bound)", worst, 1)
    assert worst <= 1, f"{name}: {worst} times its bound"


def decays(H, seed=0):
    """Between 1/2 and 1, both among them from three heads on."""
    g = 1 - 2.0 ** -(1 + 8 * torch.rand(H, generator=torch.Generator().manual_seed(seed)))
    if H > 1:
        g[-1] = 1.0
    if H > 2:
        g[0] = 0.5
    return g


class Problem:
    def __init__(self, shape, dtype, seed, start=True, lens=None):
        B, L, H, Hk, D, Dv = self.shape = shape
        self.g = torch.Generator().manual_seed(seed)
        r = lambda *s, dtype=dtype: torch.randn(s, generator=self.g).to(dtype)  # noqa: E731
        self.dtype, self.r = dtype, r
        self.q, self.k, self.v, self.do = r(B, L, H, D), r(B, L, Hk, D), r(B, L, Hk, Dv), r(B, L, H, Dv)
        self.S0 = r(B, H, D, Dv, dtype=F32) if start else None
        self.dS = r(B, H, D, Dv, dtype=F32) if start else None
        self.gamma, self.scale = decays(H, seed), 0.3
        self.lens = lens
        self.K = 2 * L + 2 * D + 64 + H // max(1, Hk)

    def host(self):
        return [n64(t) for t in (self.q, self.k, self.v)]

    def dev(self):
        return [t.cuda() for t in (self.q, self.k, self.v)]

    def kw(self):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        lens = None if self.lens is None else torch.tensor(self.lens, dtype=torch.int32).cuda()
        return {"gamma": self.gamma, "scale": self.scale, "S0": c(self.S0), "lens": lens}

    def ref(self, mag=False):
        return ort.forward(*self.host(), n64(self.gamma), self.scale, n64(self.S0), self.lens, mag=mag)

    def grads(self, mag=False):
        return ort.backward(*self.host(), n64(self.do), n64(self.gamma), self.scale, n64(self.S0), n64(self.dS),
                            self.lens, mag=mag)


# (B, L, H, Hk, D, Dv): one token, lengths around the chunks of 64 and 128, both
# widths of the tensor-core kernel and mixed ones, shared heads, odd widths,
# few heads over many tokens (parts), one head
SHAPES = [
    (1, 1, 1, 1, 64, 64), (2, 3, 2, 1, 128, 128), (1, 63, 3, 3, 64, 128), (2, 64, 2, 2, 128, 64),
    (1, 65, 4, 2, 64, 64), (3, 127, 2, 2, 128, 128), (1, 128, 3, 1, 128, 64), (1, 129, 2, 2, 64, 64),
    (2, 257, 6, 2, 128, 128), (1, 1111, 2, 1, 64, 64), (1, 1500, 1, 1, 128, 128), (5, 200, 8, 4, 64, 64),
    (2, 150, 2, 2, 8, 8), (1, 130, 3, 3, 96, 40), (1, 300, 2, 1, 256, 256), (2, 70, 2, 2, 32, 160),
    (1, 400, 2, 2, 128, 192), (1, 520, 4, 1, 64, 32),
]


@DT
@pytest.mark.parametrize("shape", SHAPES, ids=sid)
def test_forward(la, dtype, shape):
    p = Problem(shape, dtype, shape[1])
    (ro, rS), (mo, mS) = p.ref(), p.ref(True)
    o, S = la.forward_retention(*p.dev(), **p.kw(), return_state=True)
    close("o", o, ro, mo, p.K, dtype, True)
    close("state", S, rS, mS, p.K, F32)
    # the same without the state, without a start
    o2 = la.forward_retention(*p.dev(), **p.kw())
    close("o alone", o2, ro, mo, p.K, dtype, True)
    p.S0 = None
    o3 = la.forward_retention(*p.dev(), **p.kw())
    close("o from zero", o3, p.ref()[0], p.ref(True)[0], p.K, dtype, True)


@DT
@pytest.mark.parametrize("shape", SHAPES, ids=sid)
def test_backward(la, dtype, shape):
    p = Problem(shape, dtype, shape[1] + 1)
    ref, mag = p.grads(), p.grads(True)
    got = la.backward_retention(*p.dev(), p.do.cuda(), **p.kw(), dS=p.dS.cuda())
    for name, x, r, m in zip(("dq", "dk", "dv"), got, ref, mag):
        close(name, x, r, m, p.K, dtype, True)
    close("dS0", got[3], ref[3], mag[3], p.K, F32)
    # without states at the ends
    p.S0 = p.dS = None
    got = la.backward_retention(*p.dev(), p.do.cuda(), gamma=p.gamma, scale=p.scale)
    assert got[3] is None
    for name, x, r, m in zip(("dq", "dk", "dv"), got, p.grads(), p.grads(True)):
        close(name + " from zero", x, r, m, p.K, dtype, True)


RAGGED = [(6, 400, 2, 1, 64, 64), (6, 400, 2, 2, 128, 128), (6, 300, 1, 1, 40, 72)]
LENS = [400, 0, 1, 257, 128, -3]


@DT
@pytest.mark.parametrize("shape", RAGGED, ids=sid)
def test_ragged(la, dtype, shape):
    """Rows behind a sequence's end: not read (NaN there), outputs left alone,
    gradients zero."""
    B, L, H, Hk, D, Dv = shape
    lens = [min(n, L) for n in LENS]
    p = Problem(shape, dtype, 5, lens=lens)
    ref, mag, gref, gmag = p.ref(), p.ref(True), p.grads(), p.grads(True)
    for b, n in enumerate(lens):
        for t in (p.q, p.k, p.v, p.do):
            t[b, max(n, 0):] = float("nan")
    out = torch.full((B, L, H, Dv), -3.0, dtype=dtype).cuda()
    o, S = la.forward_retention(*p.dev(), **p.kw(), out=out, return_state=True)
    for b, n in enumerate(lens):
        assert (o[b, max(n, 0):] == -3).all()
        o[b, max(n, 0):] = 0
    close("ragged o", o, ref[0], mag[0], p.K, dtype, True)
    close("ragged state", S, ref[1], mag[1], p.K, F32)
    got = la.backward_retention(*p.dev(), p.do.cuda(), **p.kw(), dS=p.dS.cuda())
    for b, n in enumerate(lens):
        for t in got[:3]:
            assert not t[b, max(n, 0):].any()
    for name, x, r, m in zip(("dq", "dk", "dv"), got, gref, gmag):
        close("ragged " + name, x, r, m, p.K, dtype, True)
    close("ragged dS0", got[3], gref[3], gmag[3], p.K, F32)


@DT
@pytest.mark.parametrize("shape", [(2, 150, 4, 2, 64, 64), (2, 150, 4, 2, 128, 128), (2, 90, 4, 2, 24, 56)], ids=sid)
def test_layouts(la, dtype, shape):
    """Slices of one projection, heads first, padded rows: the dense results."""
    B, L, H, Hk, D, Dv = shape
    p = Problem(shape, dtype, 9)
    q, k, v = p.dev()
    do = p.do.cuda()
    kw = p.kw()
    o = la.forward_retention(q, k, v, **kw)
    grads = la.backward_retention(q, k, v, do, **kw, dS=p.dS.cuda())
    joint = torch.cat([t.flatten(2) for t in (q, k, v)], -1).split([H * D, Hk * D, Hk * Dv], -1)
    joint = [t.unflatten(-1, (-1, w)) for t, w in zip(joint, (D, D, Dv))]
    first = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    padded = [torch.nn.functional.pad(t, (0, 8, 0, 1, 0, 2))[:, :L, :n, :w]
              for t, n, w in ((q, H, D), (k, Hk, D), (v, Hk, Dv))]
    tokens_first = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    for args in (joint, first, padded, tokens_first):
        assert torch.equal(la.forward_retention(*args, **kw), o)
        out = torch.empty(B, H, L, Dv, dtype=dtype, device="cuda").transpose(1, 2)
        assert la.forward_retention(*args, **kw, out=out) is out and torch.equal(out, o)
        for x, y in zip(la.backward_retention(*args, do.transpose(1, 2).contiguous().transpose(1, 2), **kw, dS=p.dS.cuda()), grads):
            assert torch.equal(x, y)


@DT
def test_zero_decay_and_none(la, dtype):
    """A decay of zero keeps the newest token alone; no decay is one."""
    p = Problem((1, 140, 2, 2, 64, 64), dtype, 3)
    p.gamma = torch.tensor([0.0, 1.0])
    (ro, rS), (mo, mS) = p.ref(), p.ref(True)
    o, S = la.forward_retention(*p.dev(), **p.kw(), return_state=True)
    close("o", o, ro, mo, p.K, dtype, True)
    close("state", S, rS, mS, p.K, F32)
    kw = p.kw()
    kw["gamma"] = 1.0
    a = la.forward_retention(*p.dev(), **kw)
    kw["gamma"] = None
    assert torch.equal(a, la.forward_retention(*p.dev(), **kw))


def test_long_decay_far(la):
    """Thousands of tokens at strong and weak decays stay finite and right."""
    p = Problem((1, 4000, 4, 4, 64, 64), BF16, 4)
    p.gamma = torch.tensor([0.5, 0.03, 0.999, 1.0])
    (ro, rS), (mo, mS) = p.ref(), p.ref(True)
    o, S = la.forward_retention(*p.dev(), **p.kw(), return_state=True)
    # log2 0.03 = -5.06: powers that matter (above 2^-40) are off by 40 2^-24 more
    close("o", o, ro, mo, p.K + 40, BF16, True)
    close("state", S, rS, mS, p.K + 40, F32)


@DT
@pytest.mark.parametrize("shape", [(1, 3000, 1, 1, 128, 128), (1, 2817, 2, 1, 64, 64), (2, 2500, 1, 1, 128, 64),
                                   (1, 2600, 1, 1, 72, 40)], ids=sid)
def test_parts(la, dtype, shape):
    """Few heads over many tokens, worked in parts that all reach the end: weak
    decays and none; ragged lengths that end in front of the last parts."""
    for gamma in (1.0, 0.9995):
        p = Problem(shape, dtype, 77, lens=[shape[1] - 5, 900][:shape[0]])
        p.gamma = torch.full((shape[2],), gamma)
        (ro, rS), (mo, mS) = p.ref(), p.ref(True)
        o, S = la.forward_retention(*p.dev(), **p.kw(), return_state=True)
        for b, n in enumerate(p.lens):
            o[b, n:] = 0
        close("parts o", o, ro, mo, p.K, dtype, True)
        close("parts state", S, rS, mS, p.K, F32)
        ref, mag = p.grads(), p.grads(True)
        got = la.backward_retention(*p.dev(), p.do.cuda(), **p.kw(), dS=p.dS.cuda())
        for name, x, r, m in zip(("dq", "dk", "dv"), got, ref, mag):
            close("parts " + name, x, r, m, p.K, dtype, True)
        close("parts dS0", got[3], ref[3], mag[3], p.K, F32)


STEPS = [(1, 2, 1, 64, 64), (3, 4, 4, 128, 128), (2, 3, 3, 8, 16), (2, 2, 1, 256, 256), (1, 3, 3, 96, 40),
         (40, 16, 8, 64, 128), (40, 16, 16, 128, 64), (30, 16, 2, 136, 200)]


@DT
@pytest.mark.parametrize("shape", STEPS, ids=sid)
def test_step(la, dtype, shape):
    B, H, Hk, D, Dv = shape
    p = Problem((B, 1, H, Hk, D, Dv), dtype, D)
    (ro, rS), (mo, mS) = p.ref(), p.ref(True)
    q, k, v = (t[:, 0] for t in p.dev())
    S = p.S0.cuda()
    o = la.decode_retention(q, k, v, S, gamma=p.gamma, scale=p.scale)
    close("step o", o, ro[:, 0], mo[:, 0], D + 16, dtype)
    close("step state", S, rS, mS, 4, F32)
    # a pool, idle rows, strided inputs
    pool = torch.randn(B + 3, H, D, Dv).cuda()
    before = pool.clone()
    slots = torch.randperm(B + 3)[:B].to(torch.int32)
    for b in range(B):
        pool[slots[b]] = p.S0[b].cuda()
    idle = B > 1
    if idle:
        before[slots[0]] = pool[slots[0]]
        slots[0], lost = (-1 if dtype == F32 else B + 3), int(slots[0])
    joint = torch.cat([t.flatten(1) for t in (q, k, v)], -1).split([H * D, Hk * D, Hk * Dv], -1)
    joint = [t.unflatten(-1, (-1, w)) for t, w in zip(joint, (D, D, Dv))]
    out = torch.full_like(o, -3.0)
    la.decode_retention(*joint, pool, gamma=p.gamma, scale=p.scale, slots=slots.cuda(), out=out)
    for b in range(B):
        if idle and b == 0:
            assert (out[0] == -3).all() and torch.equal(pool[lost], before[lost])
            continue
        assert torch.equal(out[b], o[b]) and torch.equal(pool[slots[b]], S[b])
        before[slots[b]] = S[b]
    assert torch.equal(pool, before)


@DT
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_then_tokens(la, dtype, D):
    """A prompt in two segments and then tokens, against one call."""
    B, L, H = 2, 300, 3
    p = Problem((B, L, H, H, D, D), dtype, 21)
    (ro, rS), (mo, mS) = p.ref(), p.ref(True)
    q, k, v = p.dev()
    kw = p.kw()
    del kw["lens"]
    o1, S = la.forward_retention(q[:, :170], k[:, :170], v[:, :170], **kw, return_state=True)
    kw["S0"] = S
    o2, S = la.forward_retention(q[:, 170:290], k[:, 170:290], v[:, 170:290], **kw, return_state=True)
    del kw["S0"]
    outs = [o1, o2]
    for t in range(290, 300):
        outs.append(la.decode_retention(q[:, t], k[:, t], v[:, t], S, **kw)[:, None])
    close("o", torch.cat(outs, 1), ro, mo, p.K, dtype, True)
    close("state", S, rS, mS, p.K, F32)


def test_empty(la):
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    S0 = torch.randn(2, 3, 64, 64, device="cuda")
    o, S = la.forward_retention(z(2, 0, 3, 64), z(2, 0, 3, 64), z(2, 0, 3, 64), S0=S0, return_state=True)
    assert o.shape == (2, 0, 3, 64) and torch.equal(S, S0)
    assert not la.forward_retention(z(2, 0, 3, 64), z(2, 0, 3, 64), z(2, 0, 3, 64), return_state=True)[1].any()
    got = la.backward_retention(z(2, 0, 3, 64), z(2, 0, 3, 64), z(2, 0, 3, 64), z(2, 0, 3, 64), S0=S0, dS=S0)
    assert torch.equal(got[3], S0)
    assert la.forward_retention(z(0, 5, 3, 64), z(0, 5, 3, 64), z(0, 5, 3, 64)).shape == (0, 5, 3, 64)
    assert la.decode_retention(z(0, 3, 64), z(0, 3, 64), z(0, 3, 64), z(0, 3, 64, 64)).shape == (0, 3, 64)


@DT
def test_captured_and_streams(la, dtype):
    """Captured calls replay with other inputs and lengths; a call on another
    stream; two graphs and an eager call interleaved."""
    p = Problem((2, 700, 2, 1, 64, 64), dtype, 31, lens=[700, 300])
    q, k, v = p.dev()
    do, dS, kw = p.do.cuda(), p.dS.cuda(), p.kw()
    forward = lambda: la.forward_retention(q, k, v, **kw, return_state=True)  # noqa: E731
    backward = lambda: la.backward_retention(q, k, v, do, **kw, dS=dS)  # noqa: E731
    side = torch.cuda.Stream()
    graphs = []
    for f in (forward, backward):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            held = f()
        graphs.append((g, held, f))
    for t in (q, k, v, do):
        t.copy_(torch.randn(t.shape, generator=p.g).to(dtype))
    kw["lens"].copy_(torch.tensor([130, 699], dtype=torch.int32))
    torch.cuda.synchronize()
    for _ in range(2):
        for g, held, f in graphs:
            for t in held:
                t.zero_()
            g.replay()
            for i, (x, y) in enumerate(zip(held, f())):
                if f is forward and i == 0:
                    for b, n in enumerate((130, 699)):
                        assert torch.equal(x[b, :n], y[b, :n])
                else:
                    assert torch.equal(x, y)
    with torch.cuda.stream(side):
        again = forward()
    side.synchronize()
    assert torch.equal(again[1], forward()[1])


# --- beams ---

def check_select(la, logits, scores, n, finished=None, eos=None):
    got = la.select_beams(logits.cuda(), scores.cuda(), n=n, finished=None if finished is None else finished.cuda(), eos=eos)
    ref = ort.select(n64(logits), n64(scores), n, None if finished is None else finished.numpy(), eos)
    assert got[1].cpu().tolist() == ref[1].tolist()
    assert got[2].cpu().tolist() == ref[2].tolist()
    s = n64(got[0])
    live = np.isfinite(ref[0])
    assert (np.isfinite(s) == live).all()
    # the score's own rounding, and the sum of exponentials: each exponential and
    # the sums of up to 32 in a thread, 8 over lanes and warps, 2^-24 each
    tol = 2.0 ** -24 * np.abs(ref[0][live]) + 64 * 2.0 ** -24
    assert (np.abs(s[live] - ref[0][live]) <= tol).all()
    return got


@DT
@pytest.mark.parametrize("shape", [(1, 1, 5, 1), (2, 3, 7, 21), (3, 4, 1000, 8), (1, 4, 8191, 4), (1, 4, 30011, 8),
                                   (70, 5, 9001, 10), (2, 16, 2047, 32), (1, 32, 333, 64), (200, 4, 64, 8)], ids=sid)
def test_select(la, dtype, shape):
    B, K, V, n = shape
    g = torch.Generator().manual_seed(V)
    logits = (torch.randn(B, K, V, generator=g) * 3).to(dtype)
    scores = torch.randn(B, K, generator=g) * 2 - 5
    check_select(la, logits, scores, n)
    finished = torch.rand(B, K, generator=g) < 0.4
    check_select(la, logits, scores, n, finished, 3)


@DT
def test_select_hard(la, dtype):
    """Equal logits, rows that offer nothing, forbidden tokens, unused beams."""
    inf, nan = float("inf"), float("nan")
    V = 5000
    flat = torch.zeros(1, 2, V, dtype=dtype)                 # all equal, over every piece's buffer
    check_select(la, flat, torch.tensor([[-1.0, -1.0]]), 16)
    check_select(la, torch.full((1, 3, V), -inf, dtype=dtype), torch.zeros(1, 3), 4)
    x = torch.randn(1, 6, V, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[0, 0, 17] = nan
    x[0, 1, 4000] = inf
    x[0, 2, :] = -inf
    x[0, 2, 7] = 1.0                                         # one allowed token
    x[0, 3, 100:] = -inf
    x[0, 5] = -inf
    x[0, 5, 9] = nan                                         # nothing but a NaN
    scores = torch.tensor([[0.0, 0.0, -30.0, -1.0, -inf, 0.0]])
    got = check_select(la, x, scores, 12)
    assert set(got[1][0].tolist()) <= {2, 3}
    got = check_select(la, x, scores, 64)
    assert got[1][0].tolist().count(2) <= 1
    # fewer continuations than asked for
    x[0, 3] = -inf
    x[0, 3, 50] = 0.0
    got = check_select(la, x, scores, 5)
    assert got[1][0].tolist() == [3, 2, -1, -1, -1]
    # values far apart and large
    y = torch.tensor([[[3e4, -3e4, 0.0] + [1e4] * 61]]).to(dtype)
    check_select(la, y, torch.tensor([[2.0]]), 3)


@DT
@pytest.mark.parametrize("V,pad", [(1001, 0), (1000, 24), (1003, 5), (64, 1)])
def test_select_rows(la, dtype, V, pad):
    """Rows off the 16-byte boundary, inside a wider tensor of NaN."""
    g = torch.Generator().manual_seed(V)
    wide = torch.full((1 + 3 * 4 * (V + pad) + 16,), float("nan")).to(dtype).cuda()
    for off in range(0, 9, 3):
        x = wide[1 + off:1 + off + 12 * (V + pad)].view(3, 4, V + pad)[..., :V]
        x.copy_(torch.randn(3, 4, V, generator=g))
        scores = torch.randn(3, 4, generator=g)
        got = la.select_beams(x, scores.cuda(), n=7)
        ref = ort.select(n64(x), n64(scores), 7)
        assert got[1].cpu().tolist() == ref[1].tolist() and got[2].cpu().tolist() == ref[2].tolist()
        wide.fill_(float("nan"))


@pytest.mark.parametrize("B,K", [(1, 1), (3, 2), (2, 4), (5, 7), (2, 16), (3, 32), (66000, 2)])
def test_reorder(la, B, K):
    """In place, over every word size; parents outside keep a beam's own."""
    g = torch.Generator().manual_seed(B + K)
    parents = torch.randint(-1, K + 1, (B, K), generator=g, dtype=torch.int32)
    big = B > 1000
    states = [torch.randn(B, K, 4 if big else 3000, generator=g), torch.randn(B * K, 3, 8, generator=g).bfloat16(),
              torch.randint(0, 9, (B, K, 5), generator=g), torch.randint(0, 9, (B, K, 7), generator=g, dtype=torch.uint8),
              torch.randn(B, K, 1, generator=g), torch.empty(B, K, 0)]
    own = torch.where((parents < 0) | (parents >= K), torch.arange(K, dtype=torch.int32), parents).long()
    rows = torch.arange(B)[:, None]
    dev = [t.cuda() for t in states]
    assert la.reorder_states(dev, parents.cuda()) is dev
    for t, d in zip(states, dev):
        want = t.view(B, K, -1)[rows, own] if t.numel() else t.view(B, K, 0)
        assert torch.equal(d.cpu().view(B, K, -1) if t.numel() else d.cpu(), want)
    one = states[0].cuda()
    la.reorder_states(one, parents.cuda())
    assert torch.equal(one, dev[0])
    # more tensors than one launch takes, some of them off the 16-byte boundary
    if not big:
        many = [torch.randn(B * K * 12 + 1, generator=g).cuda() for _ in range(70)]
        views = [t[i % 2:B * K * 12 + i % 2].view(B, K, 12) for i, t in enumerate(many)]
        want = [t[rows.cuda(), own.cuda()] for t in views]
        la.reorder_states(views, parents.cuda())
        assert all(torch.equal(a, b) for a, b in zip(views, want))


@DT
def test_beam_search(la, dtype):
    """Together as they are used: a prompt, then tokens with beams whose states,
    convolution states and tokens follow the selection, captured as a graph and
    eager, against a search that recomputes every beam from its tokens in fp64."""
    B, K, H, D, V, steps = 2, 3, 2, 64, 50, 6
    g = torch.Generator().manual_seed(11)
    emb = torch.randn(V, 3 * H * D, generator=g).to(dtype)
    head = (torch.randn(H * D, V, generator=g) * 0.02).to(dtype)
    prompt = torch.randint(3, V, (B, 140), generator=g)
    gamma = decays(H, 5)
    emb_d, head_d = emb.cuda(), head.cuda()

    def split(x):
        return [t.unflatten(-1, (H, D)) for t in x.split(H * D, -1)]

    _, S = la.forward_retention(*split(emb_d[prompt.cuda()]), gamma=gamma, scale=0.1, return_state=True)
    S = S.repeat_interleave(K, 0)
    tokens = torch.zeros(B, K, steps, dtype=torch.int32, device="cuda")
    scores = torch.tensor([[0.0] + [-float("inf")] * (K - 1)] * B, device="cuda")
    last = prompt[:, -1:].expand(B, K).cuda().to(torch.int32).contiguous()
    at = torch.zeros(1, dtype=torch.long, device="cuda")

    def step():
        o = la.decode_retention(*split(emb_d[last.long().flatten()]), S, gamma=gamma, scale=0.1)
        logits = (o.flatten(1).float() @ head_d.float()).view(B, K, V)
        s, parents, chosen = la.select_beams(logits, scores)
        la.reorder_states([S, tokens], parents)
        scores.copy_(s)
        last.copy_(chosen.clamp(min=0))
        tokens.index_copy_(2, at, chosen[..., None])
        at.add_(1)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps - 1):
        graph.replay()
    # fp64, from the tokens alone
    e, w = n64(emb), n64(head)
    for b in range(B):
        beams = [(0.0, [])]
        for _ in range(steps):
            cand = []
            for s, toks in beams:
                seq = np.concatenate([prompt[b].numpy(), prompt[b, -1:].numpy(), np.array(toks, dtype=np.int64)])
                x = e[seq][None]
                q, k, v = (x[..., i * H * D:(i + 1) * H * D].reshape(1, -1, H, D) for i in range(3))
                o = ort.forward(q, k, v, n64(gamma), 0.1)[0][0, -1].reshape(-1)
                z = o @ w
                lp = s + z - (z.max() + np.log(np.exp(z - z.max()).sum()))
                cand += [(lp[t], toks + [t]) for t in range(V)]
            beams = sorted(cand, key=lambda c: -c[0])[:K]
        got = [(float(scores[b, i]), tokens[b, i].tolist()) for i in range(K)]
        # bf16 rounds outputs of size about 1: their step times the head's weights
        slack = 1e-4 if dtype == F32 else 0.05
        for (gs, gt), (rs, rt) in zip(got, beams):
            assert abs(gs - rs) < slack * steps
            assert dtype == BF16 or gt == rt


# --- further uses ---

# more than 128 features (two roles whose outputs are added) on both kernels
BROAD = [(2, 260, 2, 1, 192, 64), (1, 140, 2, 2, 256, 64), (2, 300, 2, 2, 64, 256), (1, 200, 2, 1, 136, 32),
         (1, 131, 1, 1, 256, 136), (1, 90, 3, 1, 200, 248)]


@DT
@pytest.mark.parametrize("shape", BROAD, ids=sid)
def test_more_features(la, dtype, shape):
    test_forward(la, dtype, shape)
    test_backward(la, dtype, shape)


@DT
@pytest.mark.parametrize("shape", [(6, 300, 2, 1, 256, 128), (6, 300, 2, 2, 136, 72)], ids=sid)
def test_more_features_ragged(la, dtype, shape):
    test_ragged(la, dtype, shape)


@DT
@pytest.mark.parametrize("shape", [(1, 2600, 1, 1, 256, 64), (1, 2600, 2, 1, 72, 200)], ids=sid)
def test_more_features_parts(la, dtype, shape):
    test_parts(la, dtype, shape)


@DT
@pytest.mark.parametrize("shape", [(2, 150, 4, 2, 256, 64), (2, 150, 2, 2, 64, 256)], ids=sid)
def test_more_features_layouts(la, dtype, shape):
    test_layouts(la, dtype, shape)


# fewer than 64 features (filled up with zeros on the tensor cores) and 128 and a few
NARROW = [(2, 300, 2, 1, 32, 32), (1, 200, 2, 2, 8, 32), (1, 260, 3, 1, 40, 64), (2, 150, 2, 1, 160, 96),
          (1, 1, 1, 1, 32, 32), (3, 129, 4, 2, 56, 128), (1, 140, 1, 1, 152, 160)]


@DT
@pytest.mark.parametrize("shape", NARROW, ids=sid)
def test_fewer_features(la, dtype, shape):
    test_forward(la, dtype, shape)
    test_backward(la, dtype, shape)


@DT
def test_fewer_features_ragged_parts_layouts(la, dtype):
    test_ragged(la, dtype, (6, 300, 2, 1, 32, 64))
    test_parts(la, dtype, (1, 2600, 1, 1, 32, 32))
    test_layouts(la, dtype, (2, 150, 4, 2, 32, 32))


@DT
@pytest.mark.parametrize("D", [64, 256])
def test_out_off_the_sectors(la, dtype, D):
    """Outputs whose rows start 8 elements off the 32-byte sectors; what lies
    between the rows stays."""
    B, L, H = 2, 200, 2
    p = Problem((B, L, H, H, D, 64), dtype, 13)
    want = la.forward_retention(*p.dev(), **p.kw())
    for off, width in ((8, 72), (8, 88), (0, 72), (16, 80)):
        room = torch.full((B, L, H, width + 8), -3.0, dtype=dtype, device="cuda")
        out = room[..., off:off + 64]
        la.forward_retention(*p.dev(), **p.kw(), out=out)
        assert torch.equal(out, want)
        out.fill_(-3.0)
        assert (room == -3).all()


@DT
@pytest.mark.parametrize("shape", [(2, 140, 2, 2, 64, 64), (1, 300, 1, 1, 40, 24)], ids=sid)
def test_zero_decay_gradients(la, dtype, shape):
    p = Problem(shape, dtype, 3)
    p.gamma = torch.zeros(shape[2])
    ref, mag = p.grads(), p.grads(True)
    got = la.backward_retention(*p.dev(), p.do.cuda(), **p.kw(), dS=p.dS.cuda())
    for name, x, r, m in zip(("dq", "dk", "dv"), got, ref, mag):
        close("zero decay " + name, x, r, m, p.K, dtype, True)
    close("zero decay dS0", got[3], ref[3], mag[3], p.K, F32)


@DT
@pytest.mark.parametrize("scale", [2.0 ** -64, -2.0 ** -20, 2.0 ** 20])
def test_scales(la, dtype, scale):
    """Scales far from one (powers of two: no rounding of their own)."""
    p = Problem((1, 150, 2, 1, 64, 64), dtype, 17)
    p.scale = scale
    (ro, _), (mo, _) = p.ref(), p.ref(True)
    close("scaled o", la.forward_retention(*p.dev(), **p.kw()), ro, mo, p.K, dtype, True)
    ref, mag = p.grads(), p.grads(True)
    got = la.backward_retention(*p.dev(), p.do.cuda(), **p.kw(), dS=p.dS.cuda())
    for name, x, r, m in zip(("dq", "dk", "dv"), got, ref, mag):
        # states of dk and dv are held divided by the scale: one rounding more
        close("scaled " + name, x, r, m, p.K + 2, dtype, True)


@pytest.mark.parametrize("shape", [(2, 150, 4, 2, 64, 128), (1, 700, 1, 1, 40, 24), (1, 100, 2, 1, 256, 64)], ids=sid)
def test_gradients_are_differences(la, shape):
    """The loss sum(o do) + sum(S dS) is linear in each input alone: its change
    along a direction is the gradient's product with it, up to the roundings of
    both, whose bounds are the outputs' own."""
    p = Problem(shape, F32, 23)
    do, dS = n64(p.do), n64(p.dS)
    grads, gmag = [n64(t) for t in la.backward_retention(*p.dev(), p.do.cuda(), **p.kw(), dS=p.dS.cuda())], p.grads(True)

    def loss():
        o, S = la.forward_retention(*p.dev(), **p.kw(), return_state=True)
        (mo, mS) = p.ref(True)
        step = (p.K + 1) * 2.0 ** -24
        return (n64(o) * do).sum() + (n64(S) * dS).sum(), step * ((mo * np.abs(do)).sum() + (mS * np.abs(dS)).sum())

    for i, name in enumerate(("q", "k", "v", "S0")):
        t = getattr(p, name)
        way = torch.randint(-1, 2, t.shape, generator=p.g).float()
        kept = t.clone()
        t.copy_(kept + way)
        up = t.clone()
        a, ea = loss()
        t.copy_(kept - way)
        moved = n64(up) - n64(t)  # as rounded
        b, eb = loss()
        t.copy_(kept)
        want = (grads[i] * moved).sum()
        bound = ea + eb + (p.K + 1) * 2.0 ** -24 * (gmag[i] * np.abs(moved)).sum()
        assert abs(a - b - want) <= bound, (name, a - b, want, bound)
        # not an empty test: the gradient's terms together exceed the worst case of the roundings
        assert bound < np.abs(grads[i] * moved).sum()


@DT
def test_offsets_beyond_32_bits(la, dtype):
    """Rows, heads and sequences more than 2^31 elements apart, and a decode whose
    places lie behind 2^31 elements of the pool."""
    B, L, H, D = 2, 130, 2, 64
    p = Problem((B, L, H, H, D, D), dtype, 19)
    o, S = la.forward_retention(*p.dev(), **p.kw(), return_state=True)
    grads = la.backward_retention(*p.dev(), p.do.cuda(), **p.kw(), dS=p.dS.cuda())
    far = (1 << 31) + (1 << 12)
    for order in ((0, 1, 2), (2, 1, 0)):  # the far stride: of sequences, of heads
        room = torch.empty(far + 5 * L * H * D * B, dtype=dtype, device="cuda")
        sizes = [(B, L, H)[i] for i in order]
        strides = [0, 0, 0]
        strides[order[0]], strides[order[1]], strides[order[2]] = far, sizes[2] * D, D
        step = L * H * D
        views = [room[i * step:].as_strided((B, L, H, D), (*strides, 1), i * step) for i in range(4)]
        for view, t in zip(views, (*p.dev(), p.do.cuda())):
            view.copy_(t)
        out = torch.empty(far + step * B, dtype=dtype, device="cuda").as_strided((B, L, H, D), (*strides, 1))
        got, gs = la.forward_retention(*views[:3], **p.kw(), out=out, return_state=True)
        assert torch.equal(got, o) and torch.equal(gs, S)
        for x, y in zip(la.backward_retention(*views[:4], **p.kw(), dS=p.dS.cuda()), grads):
            assert torch.equal(x, y)
        del room, views, got, out
    slots = torch.tensor([(1 << 19) + 3, 2, (1 << 19) + 5], dtype=torch.int32)
    p = Problem((3, 1, 1, 1, 64, 64), dtype, 2)
    q, k, v = (t[:, 0] for t in p.dev())
    near = p.S0.cuda()
    want = la.decode_retention(q, k, v, near, gamma=p.gamma, scale=p.scale)
    pool = torch.empty((1 << 19) + 6, 1, 64, 64, device="cuda")
    pool[slots.long().cuda()] = p.S0.cuda()
    got = la.decode_retention(q, k, v, pool, gamma=p.gamma, scale=p.scale, slots=slots.cuda())
    assert torch.equal(got, want) and torch.equal(pool[slots.long().cuda()], near)


@DT
def test_two_at_once(la, dtype):
    """Calls on two streams at the same time, each with its own workspace, and the
    same calls again: the same bits."""
    ps = [Problem((1, 3000, 2, 1, 128, 128), dtype, s) for s in (1, 2)]
    logits = [torch.randn(8, 4, 30011, device="cuda").to(dtype) for _ in ps]
    scores = torch.randn(8, 4, device="cuda")
    args = [(p.dev(), p.do.cuda(), p.kw(), p.dS.cuda()) for p in ps]

    def all_of(i):
        x, do, kw, dS = args[i]
        return (*la.forward_retention(*x, **kw, return_state=True), *la.backward_retention(*x, do, **kw, dS=dS),
                *la.select_beams(logits[i], scores))

    alone = [all_of(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [None, None]
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = all_of(i)
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@DT
def test_beams_captured(la, dtype):
    """A selection and the reordering after it, captured twice and replayed with
    other inputs, interleaved with eager calls."""
    B, K, V = 5, 4, 20011
    g = torch.Generator().manual_seed(8)
    logits, scores = torch.randn(B, K, V, generator=g).to(dtype).cuda(), torch.randn(B, K, generator=g).cuda()
    finished = torch.zeros(B, K, dtype=torch.bool, device="cuda")
    states = [torch.randn(B, K, 40, 64, generator=g).cuda(), torch.randn(B * K, 7, generator=g).to(dtype).cuda()]
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = la.select_beams(logits, scores, finished=finished, eos=2)
            la.reorder_states(states, held[1])
        graphs.append((graph, held))
    for turn in range(4):
        logits.copy_(torch.randn(B, K, V, generator=g).to(dtype))
        finished.copy_(torch.rand(B, K, generator=g) < 0.3)
        before = [t.clone() for t in states]
        graph, held = graphs[turn % 2]
        graph.replay()
        want = check_select(la, logits.cpu(), scores.cpu(), K, finished.cpu(), 2)
        assert all(torch.equal(x, y) for x, y in zip(held, want))
        la.reorder_states(before, want[1])
        assert all(torch.equal(x, y) for x, y in zip(states, before))


def test_select_largest(la):
    """The most beams and places; one token; a vocabulary of a million."""
    g = torch.Generator().manual_seed(4)
    check_select(la, torch.randn(2, 32, 2000, generator=g), torch.randn(2, 32, generator=g), 64)
    check_select(la, torch.zeros(3, 1, 1), torch.zeros(3, 1), 1)
    check_select(la, torch.randn(1, 2, 1 << 20, generator=g), torch.randn(1, 2, generator=g), 64)
    check_select(la, torch.randn(1, 1, 64, generator=g), torch.zeros(1, 1), 64)


@DT
@pytest.mark.parametrize("B,K,V,n", [(3, 4, 1001, 9), (1, 4, 131071, 8), (1, 8, 5003, 40), (80, 4, 9001, 9), (2, 32, 63, 64)])
def test_select_equal_rows(la, dtype, B, K, V, n):
    """Beams of equal scores that hold the same logits: equal continuations go in the
    order of the beams wherever their rows lie relative to a 16-byte boundary, and
    the scores' bits do not depend on where the logits lie or how far apart the rows
    are."""
    g = torch.Generator().manual_seed(V)
    row, scores = torch.randn(B, 1, V, generator=g) * 3, torch.randn(B, 1, generator=g).expand(B, K).contiguous()
    logits = row.expand(B, K, V).to(dtype)
    want = check_select(la, logits.contiguous(), scores, n)
    for off, pad in ((0, 1), (1, 0), (2, 3), (3, 8), (5, 2), (7, 5)):
        wide = torch.full((off + B * K * (V + pad),), float("nan"), dtype=dtype, device="cuda")
        x = wide[off:].view(B, K, V + pad)[..., :V]
        x.copy_(logits)
        got = la.select_beams(x, scores.cuda(), n=n)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (off, pad)


@DT
@pytest.mark.parametrize("B,K,V,n", [(1, 4, 333, 7), (2, 3, 5003, 40), (80, 4, 9001, 8)])
def test_select_rows_of_the_lowest_value(la, dtype, B, K, V, n):
    """A row whose logits are all masked with the type's lowest value, or all as large
    as the type goes, is a uniform one: its scores are those of zeros."""
    g = torch.Generator().manual_seed(V)
    scores = torch.randn(B, K, generator=g)
    flat = torch.zeros(B, K, V, dtype=dtype)
    want = check_select(la, flat, scores, n)
    for value in (torch.finfo(dtype).min, torch.finfo(dtype).max, -1e30, 3e4):
        got = la.select_beams(torch.full_like(flat, value).cuda(), scores.cuda(), n=n)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), value
    # a masked row beside others, masked values among a row's own
    x = (torch.randn(B, K, V, generator=g) * 3).to(dtype)
    x[:, 1] = torch.finfo(dtype).min
    x[:, 2, ::3] = torch.finfo(dtype).min
    got = la.select_beams(x.cuda(), scores.cuda(), n=n)
    alike = x.clone()
    alike[:, 1] = 0
    ref = check_select(la, alike, scores, n)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@DT
@pytest.mark.parametrize("B,K,V,n", [(1, 32, 100, 64), (2, 32, 5000, 64), (1, 20, 70001, 7), (80, 4, 9001, 8), (80, 4, 9001, 64)])
def test_select_more_ties_than_buffers(la, dtype, B, K, V, n):
    """Equal logits in all beams: more candidates than the joining pass ranks at once
    (lists in and beyond shared memory), more values in a piece than it collects
    (short and long pieces, few and many places); beams that have ended, rows that
    offer nothing and beams without a score among them."""
    flat = torch.full((B, K, V), 0.5, dtype=dtype)
    scores = torch.full((B, K), -2.0)
    check_select(la, flat, scores, n)
    finished = torch.zeros(B, K, dtype=torch.bool)
    finished[:, 1] = True
    flat[:, 2] = float("-inf")
    flat[0, 0, V // 2] = 0.75                        # one that is ahead, and one behind
    flat[0, 0, 3] = 0.25
    scores[:, 3] = float("-inf")
    check_select(la, flat, scores, n, finished, V - 1)
    check_select(la, torch.full((B, K, V), torch.finfo(dtype).min, dtype=dtype), scores, n)


def paired(g, *shape):
    """fp32 values that differ by up to 2^-9 within each 2 x 2 block of their last two
    dimensions: the first bf16 values of a pair are equal or a step apart."""
    *lead, a, b = shape
    base = (1 + torch.rand(*lead, a // 2, b // 2, generator=g)) * (2 * torch.randint(0, 2, (*lead, a // 2, b // 2), generator=g) - 1)
    wide = base.repeat_interleave(2, -2).repeat_interleave(2, -1)
    return wide * (1 + (2 * torch.rand(shape, generator=g) - 1) * 2.0 ** -9)


def differences(g, B, L, H, W):
    """Rows of bf16 that read the difference of one pair of a state's rows."""
    x = torch.zeros(B, L, H, W // 2, 2)
    v = torch.randn(B, L, H, generator=g)
    pair = torch.arange(L) % (W // 2)
    x[:, torch.arange(L), :, pair, 0] = v.permute(1, 0, 2)
    x[:, torch.arange(L), :, pair, 1] = -v.permute(1, 0, 2)
    return x.view(B, L, H, W).to(BF16)


@pytest.mark.parametrize("shape", [(1, 300, 2, 2, 64, 64), (2, 300, 2, 2, 128, 128), (1, 400, 4, 2, 128, 64),
                                   (1, 3000, 2, 2, 64, 64), (1, 300, 2, 1, 256, 64), (1, 300, 2, 1, 64, 256),
                                   (1, 300, 2, 2, 40, 32)], ids=sid)
def test_both_values_of_a_state(la, shape):
    """The states of the tensor-core kernel are sums of two bf16 values.  Here nothing
    but a state enters (no k, v or no q, dO: no weight or decayed row is rounded) and
    its rows are read as differences in which the first values nearly cancel, so
    that what is left of the bound is 2^-16 of the state (2^-8 of what the first
    value leaves, itself 2^-8), fp32 sums and the output's own rounding.  A state of
    one value, or with the second of another chunk, is many times beyond it."""
    B, L, H, Hk, D, Dv = shape
    g = torch.Generator().manual_seed(D + Dv + L)
    zk, zv = torch.zeros(B, L, Hk, D, dtype=BF16), torch.zeros(B, L, Hk, Dv, dtype=BF16)
    zq, zo = torch.zeros(B, L, H, D, dtype=BF16), torch.zeros(B, L, H, Dv, dtype=BF16)
    q, do = differences(g, B, L, H, D), differences(g, B, L, H, Dv)
    k, v = differences(g, B, L, Hk, D), differences(g, B, L, Hk, Dv)
    S = paired(g, B, H, D, Dv)
    gamma, scale = torch.tensor([1.0] + [1 - 2.0 ** -8] * (H - 1)), 0.3
    K = 2 * L + 2 * D + 2 * Dv + 64 + H // Hk
    c = lambda *ts: [t.cuda() for t in ts]  # noqa: E731
    rounded = S.to(BF16).float()

    def check(name, got, call):
        ref, mag, one = call(S, False), call(S, True), call(rounded, False)
        tol = torch.finfo(BF16).eps / 2 * np.abs(ref) + (K * 2.0 ** -24 + 2.0 ** -16) * mag + 1e-37
        worst = float((np.abs(n64(got) - ref) / tol).max())
        record(f"retention {name} of a state alone bfloat16 (share of its bound)", worst, 1)
        assert (np.abs(one - ref) / tol).max() > 8, "the first value alone has to be beyond the bound"
        assert worst <= 1, f"{name}: {worst} times its bound"

    r = lambda i, *a: lambda S, mag: ort.backward(*map(n64, a), n64(gamma), scale, *(n64(s) for s in ((S, None) if i == 0 else (None, S))), mag=mag)[i]  # noqa: E501,E731
    check("o", la.forward_retention(*c(q, zk, v), gamma, scale, S.cuda()),
          lambda S, mag: ort.forward(n64(q), n64(zk), n64(v), n64(gamma), scale, n64(S), mag=mag)[0])
    check("dq", la.backward_retention(*c(zq, k, zv, do), gamma, scale, S.cuda())[0], r(0, zq, k, zv, do))
    dq, dk, dv, _ = la.backward_retention(*c(zq, k, v, zo), gamma, scale, dS=S.cuda())
    check("dk", dk, r(1, zq, k, v, zo))
    check("dv", dv, r(2, zq, k, v, zo))


def nodes(call):
    """(launches, allocations) of a call, from the graph that it is captured into."""
    import ctypes
    call()  # kernels are loaded outside the capture
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        out = call()  # noqa: F841
    cu, count = ctypes.CDLL("libcuda.so.1"), ctypes.c_size_t(0)
    raw = ctypes.c_void_p(graph.raw_cuda_graph())
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(count)) == 0
    all_nodes = (ctypes.c_void_p * count.value)()
    assert cu.cuGraphGetNodes(raw, all_nodes, ctypes.byref(count)) == 0
    kinds = []
    for node in all_nodes:
        kind = ctypes.c_int(-1)
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        kinds.append(kind.value)
    return kinds.count(0), kinds.count(10)  # kernel, memory allocation


def test_no_records_that_nothing_reads(la):
    """Sequences of one part: a record is kept for a returned state of the tensor-core
    kernel alone, and no pass that sums states runs for roles without one."""
    def run(shape, dtype, backward, S0=True):
        B, L, H, Hk, D, Dv = shape
        p = Problem(shape, dtype, 1, start=S0)
        q, k, v, do = *p.dev(), p.do.cuda()
        kw = p.kw()
        if backward:
            return nodes(lambda: la.backward_retention(q, k, v, do, **kw))
        out, S = torch.empty_like(do), torch.empty(B, H, D, Dv, device="cuda")
        return nodes(lambda: la.forward_retention(q, k, v, **kw, out=out, S=S))

    wide = (2, 60, 200, 200, 64, 64)
    assert run(wide, F32, False) == (1, 0)
    assert run(wide, F32, True) == (1, 0)
    assert run((2, 60, 4, 4, 96, 40), BF16, False) == (1, 0)         # on CUDA cores
    assert run((2, 300, 4, 4, 64, 64), BF16, False) == (2, 1)        # the state's pass and the outputs'
    assert run((2, 300, 4, 4, 128, 64), BF16, True) == (3, 1)        # dq and dk of 64 features: no states to sum
    assert run((2, 300, 4, 4, 128, 64), BF16, True, S0=False) == (2, 0)
