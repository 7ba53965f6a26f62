"""Cases and plain forms of retention (linear attention with a decay for each head) and of beam search over its states.

Five calls of two kinds, each as its user makes it:

  retention   o_t = scale q_t S_t, S_t = gamma_h S_(t-1) + k_t v_t^T: a prompt (with its final state), one token on a
              pool of states, the backward pass
  select      the best continuations over beams and vocabulary
  reorder     the beams' states after a selection, in place

``own`` false: elementary torch operations in 32 bits (64 for the beams' scores), rounded once at the end.  ``own``
true: the library's calls.
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}
F32 = torch.float32


# --------------------------------------------------------------------------- cases

def _retention(name, mode, dtype, B, L, H, D, Dv, Hk=None, ragged=False, start=False, state=False, heads_first=False):
    return {"name": name, "op": "retention", "mode": mode, "dtype": dtype, "B": B, "L": L, "H": H, "Hk": Hk or H, "D": D,
            "Dv": Dv, "ragged": ragged, "start": start, "state": state, "heads_first": heads_first}


def _select(name, dtype, B, K, V, n, finished=True):
    return {"name": name, "op": "select", "dtype": dtype, "B": B, "K": K, "V": V, "n": n, "finished": finished}


def _reorder(name, B, K, layers, H, D, Dv, T):
    return {"name": name, "op": "reorder", "B": B, "K": K, "layers": layers, "H": H, "D": D, "Dv": Dv, "T": T}


def listed():
    return [
        # training: the forward pass of one layer over two sequences of 16384 tokens
        _retention("retention prompt", "forward", "bfloat16", 2, 16384, 16, 128, 128),
        # serving: one long prompt with its final state, queries of 8 heads over 4 heads of keys and values
        _retention("retention long state", "forward", "bfloat16", 1, 65536, 8, 128, 128, 4, state=True),
        # serving: a ragged batch that continues from cached states, narrow heads, tensors laid out heads first
        _retention("retention ragged", "forward", "bfloat16", 4, 4095, 8, 64, 64, ragged=True, start=True, state=True,
                   heads_first=True),
        # fp32, keys and values of different widths
        _retention("retention fp32", "forward", "float32", 2, 2047, 8, 64, 128, start=True, state=True),
        # the training step of a narrow layer
        _retention("retention backward", "backward", "bfloat16", 4, 4096, 8, 64, 64),
        # the training step of a wide layer over a segment of a longer sequence: gradients of the states at its ends
        _retention("retention backward ends", "backward", "bfloat16", 1, 4095, 16, 128, 128, 8, start=True),
        # one token of each of 256 sequences in serving
        _retention("retention step 256", "step", "bfloat16", 256, 1, 32, 128, 128),
        # one token of one sequence: the latency of a chat's decode
        _retention("retention step 1", "step", "bfloat16", 1, 1, 16, 128, 128),
        # one selection for 256 requests with four beams
        _select("select 256", "bfloat16", 256, 4, 32000, 8),
        # one request with four beams over a wide vocabulary of odd size
        _select("select 1", "float32", 1, 4, 131071, 4),
        # 32 requests' beams, two layers' states and their tokens so far
        _reorder("reorder 32", 32, 4, 2, 16, 128, 128, 512),
        # one request's beams in a small model
        _reorder("reorder 1", 1, 4, 4, 8, 64, 64, 127),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["retention", "retention", "retention", "select", "reorder"])
    if op == "retention":
        mode = rng.choice(["forward", "forward", "backward", "step"])
        dtype = rng.choice(["bfloat16", "bfloat16", "bfloat16", "float32"])
        D, Dv = rng.choice([(64, 64), (64, 128), (128, 64), (128, 128), (128, 128), (128, 256), (32, 32), (96, 40), (256, 256)])
        H = rng.randint(1, 32)
        Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0 and h * 8 >= H])
        if mode == "step":
            B = max(1, min(_log(rng, 1, 256), (1 << 27) // (H * D * Dv)))
            c = _retention("", mode, dtype, B, 1, H, D, Dv, Hk, heads_first=False)
        else:
            # fp32 and uncommon widths stay on the CUDA cores
            most = 8.5e9 if dtype == "bfloat16" and D in (64, 128) and Dv in (64, 128) else 2e9
            B = rng.randint(1, 8)
            L = max(1, min(_log(rng, 1, 65536), int(most / (3 if mode == "backward" else 1) / (B * H * D * Dv))))
            ragged = mode == "forward" and rng.random() < 0.4
            c = _retention("", mode, dtype, B, L, H, D, Dv, Hk, ragged, rng.random() < 0.5,
                           mode == "forward" and rng.random() < 0.5, rng.random() < 0.3)
    elif op == "select":
        K = rng.randint(1, 16)
        V = _log(rng, 64, 131072)
        B = max(1, min(_log(rng, 1, 256), int(3.2e7 / (K * V))))
        c = _select("", rng.choice(["bfloat16", "float32"]), B, K, V, rng.choice([K, 2 * K]), rng.random() < 0.6)
    else:
        K = rng.randint(2, 16)
        H, D, Dv = rng.randint(1, 16), rng.choice([32, 64, 128]), rng.choice([40, 64, 128])
        layers = rng.randint(1, 8)
        B = max(1, min(_log(rng, 1, 64), int(6.7e7 / (K * layers * H * D * Dv))))
        c = _reorder("", B, K, layers, H, D, Dv, _log(rng, 1, 4096))
    del c["name"]
    return c


def _lens(case):
    """Tokens of each sequence: all of them, or fewer from one to the next where the batch is ragged."""
    B, L = case["B"], case["L"]
    return [L - (b * L) // B if case["ragged"] else L for b in range(B)]


# --------------------------------------------------------------------------- inputs

EOS = 2


def _gammas(H):
    """Decays from 1 - 2^-5 on, with memories that grow from head to head."""
    h = torch.arange(H, dtype=torch.float64)
    return (1 - 2.0 ** (-5 - h * min(0.25, 8 / max(1, H)))).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def randn(*shape, scale=1.0, dtype=F32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case}
    B = case["B"]
    if case["op"] == "retention":
        t = DTYPES[case["dtype"]]
        L, H, Hk, D, Dv = (case[n] for n in ("L", "H", "Hk", "D", "Dv"))
        s["gamma"] = _gammas(H)  # a host tensor, as a layer keeps its constants
        s["scale"] = D ** -0.5
        widths = (H * D, Hk * D, Hk * Dv)
        tokens = (B,) if case["mode"] == "step" else (B, L)
        if case["heads_first"]:  # as the other forms of attention take them: read through transposed views
            s["q"], s["k"], s["v"] = (randn(B, n, L, w, dtype=t).transpose(1, 2) for n, w in ((H, D), (Hk, D), (Hk, Dv)))
        else:  # slices of one projection's output
            q, k, v = randn(*tokens, sum(widths), dtype=t).split(widths, -1)
            s["q"], s["k"], s["v"] = q.unflatten(-1, (H, D)), k.unflatten(-1, (Hk, D)), v.unflatten(-1, (Hk, Dv))
        if case["mode"] == "step":
            # a pool with room for more sequences than decode now, and the places of these
            pool = B + max(1, B // 4)
            s["S"] = randn(pool, H, D, Dv, scale=4.0)
            s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:B].to(torch.int32)
        else:
            s["S0"] = randn(B, H, D, Dv, scale=4.0) if case["start"] else None
            s["lens"] = s["out"] = None
            if case["ragged"]:
                s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
                s["out"] = torch.full((B, L, H, Dv), -3.0, dtype=t, device="cuda")
        if case["mode"] == "backward":
            s["do"] = randn(B, L, H, Dv, dtype=t)
            s["dS"] = randn(B, H, D, Dv) if case["start"] else None
    elif case["op"] == "select":
        K, V = case["K"], case["V"]
        # a few likely tokens above the rest; in bf16 many logits are equal
        x = randn(B, K, V, scale=2.0)
        likely = torch.randint(0, V, (B, K, 12), generator=g, device="cuda")
        s["logits"] = x.scatter_add_(2, likely, 6 + 2 * randn(B, K, 12)).to(DTYPES[case["dtype"]])
        s["scores"] = torch.sort(randn(B, K, scale=2.0) - 8, descending=True)[0]
        s["finished"] = torch.rand(B, K, generator=g, device="cuda") < 0.15 if case["finished"] else None
    else:
        K, H, D, Dv, T = (case[n] for n in ("K", "H", "D", "Dv", "T"))
        s["states"] = [randn(B, K, H, D, Dv) for _ in range(case["layers"])]
        # the convolution states of bf16 layers and the tokens so far
        s["states"] += [randn(B, K, 3, H * D, dtype=torch.bfloat16) for _ in range(case["layers"])]
        s["states"].append(torch.randint(0, 32000, (B, K, T), generator=g, device="cuda", dtype=torch.int32))
        s["parents"] = torch.randint(0, K, (B, K), generator=g, device="cuda", dtype=torch.int32)
    return s


# --------------------------------------------------------------------------- plain forms

CHUNK = 128


def _heads(t, H):
    """[B, L, Hk, w] as [B, H, L, w] in 32 bits, each head of it for its share of the H heads."""
    return t.float().transpose(1, 2).repeat_interleave(H // t.shape[2], 1)


def _chunked(x, y, w, lg, start, shift):
    """o_i = sum_(j <= i) g^(i-j) (x_i . y_j) w_j + g^(i+shift) x_i start, by chunks; [B, H, L, .], lg = log2 g [H].

    ``start`` is the state in front ([B, H, Dx, Dw] or None)."""
    B, H, L, Dx = x.shape
    C = min(CHUNK, L)
    n = -(-L // C)
    x, y, w = (torch.nn.functional.pad(t, (0, 0, 0, n * C - L)).view(B, H, n, C, -1) for t in (x, y, w))
    i = torch.arange(C, device=x.device, dtype=F32)
    lg = lg.view(1, H, 1, 1, 1)
    far = i[:, None] - i
    p = (x @ y.transpose(-1, -2)) * torch.where(far >= 0, torch.exp2(far * lg), 0.0)
    o = p @ w
    # what each chunk adds to the state at its end, and with it the state in front of each chunk
    add = (y * torch.exp2((C - 1 - i)[:, None] * lg)).transpose(-1, -2) @ w
    c = torch.arange(n, device=x.device, dtype=F32)
    back = c[:, None] - 1 - c
    m = torch.where(back >= 0, torch.exp2(back * C * lg[..., 0]), 0.0)  # [1, H, n, n]
    front = (m @ add.flatten(3)).view(add.shape)
    o += (x * torch.exp2((i + 1)[:, None] * lg)) @ front
    o = o.view(B, H, n * C, -1)[:, :, :L]
    if start is not None:
        t = torch.arange(L, device=x.device, dtype=F32) + shift
        o = o + (x.view(B, H, n * C, Dx)[:, :, :L] * torch.exp2(t[:, None] * lg[..., 0])) @ start
    return o


def _ended(y, w, lg, ends, start):
    """sum_j g^ends_j y_j^T w_j (a weight of zero where ends < 0), with g^whole start added: start is (state, whole)."""
    weight = torch.where(ends >= 0, torch.exp2(ends * lg.view(-1, 1)), 0.0)  # [B or 1, H, L]
    s = (y * weight[..., None]).transpose(-1, -2) @ w
    if start is not None:
        s = s + start[0] * torch.exp2(start[1] * lg.view(1, -1))[..., None, None]
    return s


def _plain_retention(s):
    case, t, scale = s["case"], s["q"].dtype, s["scale"]
    H, Hk, L = case["H"], case["Hk"], case["L"]
    if case["mode"] == "step":
        g = s["gamma"].cuda()
        q, k, v = s["q"].float(), s["k"].float().repeat_interleave(H // Hk, 1), s["v"].float().repeat_interleave(H // Hk, 1)
        at = s["slots"].long()
        S = s["S"][at] * g[:, None, None] + k[..., None] * v[..., None, :]
        s["S"][at] = S
        return {"o": ((q[..., None] * S).sum(-2) * scale).to(t), "S": s["S"]}
    lg = torch.log2(s["gamma"].double()).float().cuda()
    q, k, v = _heads(s["q"], H), _heads(s["k"], H), _heads(s["v"], H)
    S0 = s["S0"]
    j = torch.arange(L, device=q.device, dtype=F32)
    if case["mode"] == "forward":
        lens = torch.full((case["B"],), L, device=q.device, dtype=F32) if s["lens"] is None else s["lens"].float()
        o = (_chunked(q, k, v, lg, S0, 1) * scale).transpose(1, 2).to(t)
        if s["lens"] is not None:
            o = torch.where((j < lens[:, None])[..., None, None], o, s["out"])
        if not case["state"]:
            return {"o": o}
        S = _ended(k, v, lg, (lens[:, None] - 1 - j)[:, None], None if S0 is None else (S0, lens[:, None]))
        return {"o": o, "S": S}
    do, dS = _heads(s["do"], H), s["dS"]
    turned = None if S0 is None else S0.transpose(-1, -2)
    ends = None if dS is None else dS / scale
    group = lambda d: d.transpose(1, 2).unflatten(2, (Hk, H // Hk)).sum(3).to(t)  # noqa: E731
    got = {"dq": (_chunked(do, v, k, lg, turned, 1) * scale).transpose(1, 2).to(t)}
    rq, rk, rv, rdo = (x.flip(2) for x in (q, k, v, do))
    got["dk"] = group(_chunked(rv, rdo, rq, lg, None if ends is None else ends.transpose(-1, -2), 0).flip(2) * scale)
    got["dv"] = group(_chunked(rk, rq, rdo, lg, ends, 0).flip(2) * scale)
    if S0 is not None:
        got["dS0"] = _ended(q * scale, do, lg, (j + 1)[None, None], (dS, torch.full((1, 1), float(L), device=q.device)))
    return got


def _plain_select(s):
    case = s["case"]
    B, K, V, n = (case[x] for x in ("B", "K", "V", "n"))
    x = s["logits"].double()
    m = x.amax(-1, keepdim=True)
    total = s["scores"].double()[..., None] + (x - m - torch.log(torch.exp(x - m).sum(-1, keepdim=True)))
    if s["finished"] is not None:  # a finished beam goes on with its end token alone, at no cost
        last = torch.arange(V, device=x.device) == EOS
        kept = torch.where(last, s["scores"].double()[..., None], -math.inf)
        total = torch.where(s["finished"][..., None], kept, total)
    best, at = torch.sort(total.view(B, K * V), dim=1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    none = torch.isneginf(best)
    return {"scores": best.float(), "parents": torch.where(none, -1, at // V).to(torch.int32),
            "tokens": torch.where(none, -1, at % V).to(torch.int32)}


def _plain_reorder(s):
    at = s["parents"].long()
    rows = torch.arange(at.shape[0], device=at.device)[:, None]
    for state in s["states"]:
        state.copy_(state[rows, at])
    return s["states"]


PLAIN = {"retention": _plain_retention, "select": _plain_select, "reorder": _plain_reorder}


# --------------------------------------------------------------------------- the library's calls

def _own_retention(s):
    import kernelized_sequence_mixing_gb300 as la
    case, more = s["case"], {"gamma": s["gamma"], "scale": s["scale"]}
    if case["mode"] == "step":
        return {"o": la.decode_retention(s["q"], s["k"], s["v"], s["S"], slots=s["slots"], **more), "S": s["S"]}
    if case["mode"] == "forward":
        got = la.forward_retention(s["q"], s["k"], s["v"], **more, S0=s["S0"], lens=s["lens"], out=s["out"],
                                   return_state=case["state"])
        return dict(zip(("o", "S"), got)) if case["state"] else {"o": got}
    got = la.backward_retention(s["q"], s["k"], s["v"], s["do"], **more, S0=s["S0"], dS=s["dS"])
    return {n: v for n, v in zip(("dq", "dk", "dv", "dS0"), got) if v is not None}


def _own_select(s):
    import kernelized_sequence_mixing_gb300 as la
    got = la.select_beams(s["logits"], s["scores"], n=s["case"]["n"], finished=s["finished"], eos=EOS)
    return dict(zip(("scores", "parents", "tokens"), got))


def _own_reorder(s):
    import kernelized_sequence_mixing_gb300 as la
    la.reorder_states(s["states"], s["parents"])
    return s["states"]


OWN = {"retention": _own_retention, "select": _own_select, "reorder": _own_reorder}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# --------------------------------------------------------------------------- work

def work(case):
    """Bytes: every input read once and every output written once.  Flops: multiplications, additions and exponentials."""
    B = case["B"]
    if case["op"] == "select":
        K, V, n = case["K"], case["V"], case["n"]
        e = 4 if case["dtype"] == "float32" else 2
        return {"bytes": B * K * (V * e + 4 + case["finished"]) + 12 * B * n, "flops": 4 * B * K * V}
    if case["op"] == "reorder":
        K, H, D, Dv = (case[x] for x in ("K", "H", "D", "Dv"))
        row = case["layers"] * (4 * H * D * Dv + 2 * 3 * H * D) + 4 * case["T"]
        # of parents drawn at random: beams that change, and beams that another one takes over
        moved, read = K - 1, K * (1 - (1 - 1 / K) ** (K - 1))
        return {"bytes": int(B * (row * (moved + read) + 4 * K)), "flops": 0}
    e = 4 if case["dtype"] == "float32" else 2
    H, Hk, D, Dv = (case[x] for x in ("H", "Hk", "D", "Dv"))
    tokens = sum(_lens(case))
    row = e * (H * (D + Dv) + Hk * (D + Dv))
    S = 4 * B * H * D * Dv
    if case["mode"] == "step":
        return {"bytes": tokens * (row + 4) + 2 * S, "flops": 5 * tokens * H * D * Dv}
    if case["mode"] == "forward":
        return {"bytes": tokens * row + S * (case["start"] + case["state"]), "flops": 4 * tokens * H * D * Dv}
    # q, k, v, do in; dq, dk, dv out
    return {"bytes": tokens * (2 * row - e * H * Dv) + 3 * S * case["start"], "flops": 12 * tokens * H * D * Dv}


# --------------------------------------------------------------------------- 64 bits

def _exact_retention(s):
    """The whole matrix of weights, head by head, rows in blocks; gradients of it written out term by term."""
    case, scale = s["case"], s["scale"]
    B, H, Hk, L, mode = (case[x] for x in ("B", "H", "Hk", "L", "mode"))
    gamma = s["gamma"].double().cuda()
    if mode == "step":
        S = s["S"].double()
        o = []
        for b, at in enumerate(s["slots"].tolist()):
            k = torch.repeat_interleave(s["k"][b].double(), H // Hk, 0)
            v = torch.repeat_interleave(s["v"][b].double(), H // Hk, 0)
            S[at] = S[at] * gamma.view(H, 1, 1) + torch.einsum("hd,he->hde", k, v)
            o.append(torch.einsum("hd,hde->he", s["q"][b].double(), S[at]) * scale)
        return {"o": torch.stack(o), "S": S}
    lens = _lens(case)
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    o = new(B, L, H, case["Dv"]) if s["out"] is None else s["out"].double()
    SN = new(B, H, case["D"], case["Dv"])
    dq, dk, dv, dS0 = new(*s["q"].shape), new(*s["k"].shape), new(*s["v"].shape), new(B, H, case["D"], case["Dv"])
    for b in range(B):
        n = lens[b]
        t = torch.arange(n, device="cuda", dtype=torch.float64)
        for h in range(H):
            g, hk = gamma[h], h // (H // Hk)
            q, k, v = s["q"][b, :n, h].double(), s["k"][b, :n, hk].double(), s["v"][b, :n, hk].double()
            S0 = s["S0"][b, h].double() if s["S0"] is not None else None
            for r in range(0, n, 2048):
                rows, upto = slice(r, min(n, r + 2048)), min(n, r + 2048)
                weight = torch.tril(g ** (t[rows, None] - t[:upto]).clamp(min=0), diagonal=r)
                if mode == "forward":
                    o[b, rows, h] = scale * ((q[rows] @ k[:upto].T * weight) @ v[:upto])
                else:
                    do = s["do"][b, rows, h].double()
                    dp = (do @ v[:upto].T) * weight * scale
                    dq[b, rows, h] += dp @ k[:upto]
                    dk[b, :upto, hk] += dp.T @ q[rows]
                    dv[b, :upto, hk] += ((q[rows] @ k[:upto].T) * weight * scale).T @ do
            ahead = g ** (t + 1)
            behind = (g ** (n - 1 - t))[:, None]
            if mode == "forward":
                SN[b, h] = (k * behind).T @ v
                if S0 is not None:
                    o[b, :n, h] += scale * ahead[:, None] * (q @ S0)
                    SN[b, h] += g ** n * S0
            elif S0 is not None:
                do, dS = s["do"][b, :, h].double(), s["dS"][b, h].double()
                dq[b, :, h] += scale * ahead[:, None] * (do @ S0.T)
                dk[b, :, hk] += behind * (v @ dS.T)
                dv[b, :, hk] += behind * (k @ dS)
                dS0[b, h] = g ** n * dS + scale * (q * ahead[:, None]).T @ do
    if mode == "forward":
        return {"o": o, "S": SN} if case["state"] else {"o": o}
    return {"dq": dq, "dk": dk, "dv": dv, "dS0": dS0} if case["start"] else {"dq": dq, "dk": dk, "dv": dv}


def _exact_select(s):
    """Request by request on the candidates that can be among the n best."""
    case = s["case"]
    B, K, V, n = (case[x] for x in ("B", "K", "V", "n"))
    scores, parents, tokens = [], [], []
    for b in range(B):
        logp = s["logits"][b].double()
        logp = logp - torch.logsumexp(logp, -1, keepdim=True)
        total = logp + s["scores"][b].double()[:, None]
        if s["finished"] is not None:
            for k in torch.nonzero(s["finished"][b]).flatten().tolist():
                total[k] = -math.inf
                total[k, EOS] = s["scores"][b, k].double()
        flat = total.flatten()
        least = torch.topk(flat, n)[0][-1]
        at = torch.nonzero((flat >= least) & ~torch.isneginf(flat)).flatten()
        order = sorted(zip((-flat[at]).tolist(), at.tolist()))[:n]
        order += [(math.inf, None)] * (n - len(order))
        scores.append([-v for v, _ in order])
        parents.append([-1 if a is None else a // V for _, a in order])
        tokens.append([-1 if a is None else a % V for _, a in order])
    as_ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"scores": torch.tensor(scores, dtype=torch.float64, device="cuda"), "parents": as_ints(parents), "tokens": as_ints(tokens)}


def _exact_reorder(s):
    parents = s["parents"].tolist()
    got = []
    for state in s["states"]:
        new = torch.stack([torch.stack([state[b, p] for p in row]) for b, row in enumerate(parents)])
        got.append(new.double() if new.is_floating_point() else new)
    return got


EXACT = {"retention": _exact_retention, "select": _exact_select, "reorder": _exact_reorder}


def exact(case, seed):
    # the weights of 65536 rows and columns take too long in 64 bits
    if case["op"] == "retention" and case["mode"] != "step":
        pairs = case["B"] * case["H"] * float(case["L"]) ** 2 * (case["D"] + case["Dv"]) * (3 if case["mode"] == "backward" else 1)
        if pairs > 5e12:
            return None
    return EXACT[case["op"]](prepare(case, seed))
