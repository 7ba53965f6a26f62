"""Cases and plain forms of the selective state space operators and of the norms around a mixing block.

Four operators, each as its user calls it:

  conv           short causal depthwise convolution ahead of the scan: a prompt, one token, the backward pass
  selective      selective state space scan: a prompt (with its final state), one token, the backward pass
  norm_gate      per-head RMS norm of a mixing form's output with its SiLU gate: forward and backward
  norm_residual  scaled residual sum and the RMS norm ahead of the next block: forward and backward

``own`` false: elementary torch operations in 32 bits, rounded once at the end.  ``own`` true: the library's calls.
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}


# --------------------------------------------------------------------------- cases

def _selective(name, mode, dtype, B, L, E, N, G=1, ragged=False, start=False, gate=True):
    return {"name": name, "op": "selective", "mode": mode, "dtype": dtype, "B": B, "L": L, "E": E, "N": N, "G": G,
            "ragged": ragged, "start": start, "gate": gate}


def _conv(name, mode, dtype, B, L, E, W=4, ragged=False, start=False):
    return {"name": name, "op": "conv", "mode": mode, "dtype": dtype, "B": B, "L": L, "E": E, "W": W, "ragged": ragged,
            "start": start}


def _gate(name, mode, dtype, B, H, L, D, heads_first=True, gate_first=False):
    return {"name": name, "op": "norm_gate", "mode": mode, "dtype": dtype, "B": B, "H": H, "L": L, "D": D,
            "heads_first": heads_first, "gate_first": gate_first}


def _residual(name, mode, dtype, R, E, scale):
    return {"name": name, "op": "norm_residual", "mode": mode, "dtype": dtype, "R": R, "E": E, "scale": scale}


def listed():
    return [
        # two prompts of 4096 tokens through one layer of a model of ordinary width
        _selective("scan prompt", "forward", "bfloat16", 2, 4096, 2048, 16),
        # a ragged batch of long prompts that continue from a cached state, in fp32, with shared B and C in two groups
        _selective("scan ragged long fp32", "forward", "float32", 3, 8191, 512, 16, 2, ragged=True, start=True),
        # the training step of the first case's layer
        _selective("scan backward", "backward", "bfloat16", 2, 4096, 2048, 16),
        # one token of each of 256 sequences in serving
        _selective("scan step 256", "step", "bfloat16", 256, 1, 4096, 16),
        # one token of one sequence: the latency of a chat's decode
        _selective("scan step 1", "step", "bfloat16", 1, 1, 2048, 16),
        # prompts ahead of the scan in a wide layer
        _conv("conv prompt", "forward", "bfloat16", 4, 4096, 4096),
        # its training step, three taps and an odd length
        _conv("conv backward", "backward", "bfloat16", 2, 4095, 2048, 3),
        # one token of each of 256 sequences
        _conv("conv step 256", "step", "bfloat16", 256, 1, 4096),
        # output stage of causal linear attention over 2 x 16384 tokens, 16 heads of 128
        _gate("norm gate heads", "forward", "bfloat16", 2, 16, 16384, 128),
        # the training step of an eight-head layer
        _gate("norm gate backward", "backward", "bfloat16", 4, 8, 4096, 64),
        # one token of each of 256 sequences between two blocks
        _residual("norm residual 256", "forward", "bfloat16", 256, 4096, 1.0),
        # training: 8191 tokens of a model that scales its blocks' outputs
        _residual("norm residual backward", "backward", "bfloat16", 8191, 2048, 0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step):
    return max(step, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["selective", "selective", "conv", "norm_gate", "norm_residual"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    if op == "selective":
        mode = rng.choice(["forward", "forward", "backward", "step"])
        G = rng.choice([1, 1, 2, 4])
        N = rng.choice([8, 16, 16, 32, 64])
        E = _width(rng, 64, 4096, 8 * G)
        if mode == "step":
            B = min(_log(rng, 1, 512), (1 << 24) // (E * N))
            c = _selective("", mode, dtype, max(1, B), 1, E, N, G, gate=rng.random() < 0.7)
        else:
            most = 1.5e8 if mode == "forward" else 0.7e8
            B = rng.randint(1, 8)
            L = max(1, min(_log(rng, 1, 16384), int(most / (B * E * N))))
            ragged = mode == "forward" and rng.random() < 0.4
            c = _selective("", mode, dtype, B, L, E, N, G, ragged, rng.random() < 0.4, rng.random() < 0.7)
    elif op == "conv":
        mode = rng.choice(["forward", "backward", "step"])
        W = rng.randint(2, 4)
        E = _width(rng, 64, 4096, 8)
        if mode == "step":
            c = _conv("", mode, dtype, _log(rng, 1, 512), 1, E, W)
        else:
            B = rng.randint(1, 8)
            L = max(1, min(_log(rng, 1, 16384), int(1.6e7 / (B * E))))
            c = _conv("", mode, dtype, B, L, E, W, mode == "forward" and rng.random() < 0.4, rng.random() < 0.4)
    elif op == "norm_gate":
        D = _width(rng, 32, 2048, 8)
        H = rng.randint(1, 32)
        B = rng.randint(1, 8)
        L = max(1, min(_log(rng, 1, 16384), int(1.6e7 / (B * H * D))))
        c = _gate("", rng.choice(["forward", "backward"]), dtype, B, H, L, D, rng.random() < 0.6, rng.random() < 0.4)
    else:
        E = _width(rng, 64, 8192, 8)
        R = max(1, min(_log(rng, 1, 16384), int(1.6e7 / E)))
        c = _residual("", rng.choice(["forward", "backward"]), dtype, R, E, rng.choice([1.0, 0.5, 0.25]))
    del c["name"]
    return c


def _lens(case):
    """Tokens of each sequence: all of them, or fewer from one to the next where the batch is ragged."""
    B, L = case["B"], case["L"]
    return [L - (b * L) // B if case["ragged"] else L for b in range(B)]


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    t = DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0, dtype=t):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    f = torch.float32
    s = {"case": case}
    if case["op"] in ("selective", "conv"):
        B, L, E = case["B"], case["L"], case["E"]
        tokens = (B,) if case["mode"] == "step" else (B, L)
        # x and z are the halves of one projection's output, as a block's input projection leaves them
        xz = randn(*tokens, 2 * E)
        if case["mode"] == "forward" and case["ragged"]:
            s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
            s["out"] = torch.full((B, L, E), -3.0, dtype=t, device="cuda")
        else:
            s["lens"] = s["out"] = None
    if case["op"] == "selective":
        N, G = case["N"], case["G"]
        # x comes from the convolution, z from the projection; B and C are slices of a second projection's output
        s["x"] = randn(*tokens, E)
        s["z"] = xz[..., E:] if case["gate"] else None
        s["dt"] = randn(*tokens, E, scale=0.5)
        step = torch.exp(rand(E) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus(dt_bias) = step
        s["A"] = -(torch.arange(1, N + 1, device="cuda", dtype=f) * (0.9 + 0.2 * rand(E, 1))).contiguous()
        s["D"] = 1.0 + randn(E, scale=0.1, dtype=f)
        bc = randn(*tokens, 2, G, N)
        s["Bm"], s["Cm"] = bc[..., 0, :, :], bc[..., 1, :, :]
        if case["mode"] == "step":
            s["h"] = randn(B, E, N, scale=0.3, dtype=f)
        else:
            s["h0"] = randn(B, E, N, scale=0.3, dtype=f) if case["start"] else None
        if case["mode"] == "backward":
            s["dy"] = randn(B, L, E)
            s["dh"] = randn(B, E, N, dtype=f) if case["start"] else None
    elif case["op"] == "conv":
        W = case["W"]
        s["x"] = xz[..., :E]
        s["w"] = (rand(E, W) * 2 - 1) / math.sqrt(W)
        s["bias"] = (rand(E) * 2 - 1) / math.sqrt(W)
        s["state"] = randn(B, W - 1, E) if case["mode"] == "step" or case["start"] else None
        if case["mode"] == "backward":
            s["dy"] = randn(B, L, E)
    elif case["op"] == "norm_gate":
        B, H, L, D = case["B"], case["H"], case["L"], case["D"]
        s["y"] = randn(*((B, H, L, D) if case["heads_first"] else (B, L, H, D)), scale=0.3)
        s["gate"] = randn(B, L, H * D)
        s["w"] = 1.0 + randn(H, D, scale=0.1, dtype=f)
        if case["mode"] == "backward":
            s["do"] = randn(B, L, H * D)
    else:
        R, E = case["R"], case["E"]
        s["w"] = 1.0 + randn(E, scale=0.1, dtype=f)
        if case["mode"] == "forward":
            s["x"], s["residual"] = randn(R, E), randn(R, E, scale=2.0)
        else:
            s["r"], s["do"], s["dr"] = randn(R, E, scale=2.0), randn(R, E), randn(R, E)
    return s


# --------------------------------------------------------------------------- plain forms

def _scan(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dim 1 from h = 0, by doubling the span of each element."""
    span = 1
    while span < a.shape[1]:
        b = torch.cat((b[:, :span], torch.addcmul(b[:, span:], a[:, span:], b[:, :-span])), 1)
        a = torch.cat((a[:, :span], a[:, span:] * a[:, :-span]), 1)
        span *= 2
    return b


def _expand(m, E):
    """[..., G, N] of the groups as [..., E, N] of the channels, in 32 bits."""
    return m.float().repeat_interleave(E // m.shape[-2], -2)


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain_selective(s):
    case, t = s["case"], s["x"].dtype
    E = case["E"]
    x, A, D = s["x"].float(), s["A"], s["D"]
    raw = s["dt"].float() + s["dt_bias"]
    dt = _softplus(raw)
    z = s["z"].float() if s["z"] is not None else None
    if case["mode"] == "step":
        h = torch.exp(dt[..., None] * A) * s["h"] + (dt * x)[..., None] * _expand(s["Bm"], E)
        y = (h * _expand(s["Cm"], E)).sum(-1) + D * x
        if z is not None:
            y = y * z * torch.sigmoid(z)
        s["h"].copy_(h)
        return {"y": y.to(t), "h": s["h"]}
    if s["lens"] is not None:  # rows behind a sequence's end leave the state as it is
        inside = (torch.arange(case["L"], device=x.device) < s["lens"][:, None])[..., None]
        dt = torch.where(inside, dt, 0.0)
    a = torch.exp(dt[..., None] * A)
    b = (dt * x)[..., None] * _expand(s["Bm"], E)
    if s["h0"] is not None:
        b[:, 0] += a[:, 0] * s["h0"]
    h = _scan(a, b)
    C = _expand(s["Cm"], E)
    y = (h * C).sum(-1) + D * x
    if case["mode"] == "forward":
        if z is not None:
            y = y * z * torch.sigmoid(z)
        y = y.to(t)
        if s["lens"] is not None:
            y = torch.where(inside, y, s["out"])
        return {"y": y, "h": h[:, -1].contiguous()}
    dy, got = s["dy"].float(), {}
    if z is not None:
        sig = torch.sigmoid(z)
        got["dz"] = (dy * y * sig * (1 + z * (1 - sig))).to(t)
        dy = dy * z * sig
    # adjoint states, from the last token back: gh[t] = C[t] dy[t] + a[t+1] gh[t+1]
    gh = dy[..., None] * C
    if s["dh"] is not None:
        gh[:, -1] += s["dh"]
    after = torch.cat((a[:, 1:], torch.zeros_like(a[:, :1])), 1)
    gh = _scan(after.flip(1), gh.flip(1)).flip(1)
    del after
    B_, L, G, N = s["Bm"].shape
    got["dC"] = (dy[..., None] * h).view(B_, L, G, E // G, N).sum(3).to(t)
    got["dB"] = (gh * (dt * x)[..., None]).view(B_, L, G, E // G, N).sum(3).to(t)
    du = (gh * _expand(s["Bm"], E)).sum(-1)
    got["dx"] = (du * dt + D * dy).to(t)
    before = torch.cat(((s["h0"] if s["h0"] is not None else torch.zeros_like(h[:, 0]))[:, None], h[:, :-1]), 1)
    da = gh * before * a
    got["dA"] = (da * dt[..., None]).sum((0, 1))
    ddt = ((da * A).sum(-1) + du * x) * torch.sigmoid(raw)
    got["ddt"] = ddt.to(t)
    got["ddt_bias"] = ddt.sum((0, 1))
    got["dD"] = (dy * x).sum((0, 1))
    if s["h0"] is not None:
        got["dh0"] = a[:, 0] * gh[:, 0]
    return got


def _plain_conv(s):
    case, t = s["case"], s["x"].dtype
    B, E, W = case["B"], case["E"], case["W"]
    step = case["mode"] == "step"
    x = s["x"][:, None] if step else s["x"]
    L = x.shape[1]
    old = s["state"] if s["state"] is not None else torch.zeros(B, W - 1, E, dtype=t, device=x.device)
    rows = torch.cat((old, x), 1)
    taps = rows.float().unfold(1, W, 1)  # [B, L, E, W]
    pre = (taps * s["w"]).sum(-1) + s["bias"]
    sig = torch.sigmoid(pre)
    if step:
        s["state"].copy_(rows[:, 1:])
        return {"y": (pre * sig)[:, 0].to(t), "state": s["state"]}
    if case["mode"] == "forward":
        y = (pre * sig).to(t)
        end = torch.full((B,), L, device=x.device)
        if s["lens"] is not None:
            end = s["lens"].long()
            y = torch.where((torch.arange(L, device=x.device) < end[:, None])[..., None], y, s["out"])
        last = end[:, None] + torch.arange(W - 1, device=x.device)
        return {"y": y, "state": rows.gather(1, last[..., None].expand(-1, -1, E))}
    dpre = s["dy"].float() * sig * (1 + pre * (1 - sig))
    edge = torch.zeros(B, W - 1, E, device=x.device)
    drows = (torch.cat((edge, dpre, edge), 1).unfold(1, W, 1) * s["w"].flip(1)).sum(-1)
    got = {"dx": drows[:, W - 1:].to(t), "dw": (dpre[..., None] * taps).sum((0, 1)), "dbias": dpre.sum((0, 1))}
    if s["state"] is not None:
        got["dstate"] = drows[:, :W - 1].to(t)
    return got


EPS = 1e-5


def _plain_gate(s):
    case, t = s["case"], s["y"].dtype
    B, H, L, D = case["B"], case["H"], case["L"], case["D"]
    y = (s["y"].transpose(1, 2) if case["heads_first"] else s["y"]).float()  # [B, L, H, D]
    g, w = s["gate"].float().view(B, L, H, D), s["w"]
    sig = torch.sigmoid(g)
    act = g * sig
    p = y * act if case["gate_first"] else y
    rstd = torch.rsqrt((p * p).mean(-1, keepdim=True) + EPS)
    n = p * rstd
    if case["mode"] == "forward":
        o = n * w if case["gate_first"] else n * w * act
        return o.to(t).reshape(B, L, H * D)
    do = s["do"].float().view(B, L, H, D)
    dact = sig * (1 + g * (1 - sig))
    if case["gate_first"]:
        dw, dn = (do * n).sum((0, 1)), do * w
    else:
        dw, dn = (do * n * act).sum((0, 1)), do * w * act
    dp = rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    if case["gate_first"]:
        dg, dy = dp * y * dact, dp * act
    else:
        dg, dy = do * n * w * dact, dp
    dy = dy.to(t)
    return {"dy": dy.transpose(1, 2).contiguous() if case["heads_first"] else dy, "dgate": dg.to(t).reshape(B, L, H * D), "dw": dw}


def _plain_residual(s):
    case, w = s["case"], s["w"]
    if case["mode"] == "forward":
        r = s["residual"].float() + case["scale"] * s["x"].float()
        o = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * w
        return {"o": o.to(s["x"].dtype), "r": r.to(s["x"].dtype)}
    t = s["r"].dtype
    r, do = s["r"].float(), s["do"].float()
    rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    n, dn = r * rstd, do * w
    d = s["dr"].float() + rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    return {"dresidual": d.to(t), "dx": (case["scale"] * d).to(t), "dw": (do * n).sum(0)}


PLAIN = {"selective": _plain_selective, "conv": _plain_conv, "norm_gate": _plain_gate, "norm_residual": _plain_residual}


# --------------------------------------------------------------------------- the library's calls

def _own_selective(s):
    import kernelized_sequence_mixing_gb300 as la
    mode = s["case"]["mode"]
    args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
    more = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"], "softplus": True}
    if mode == "step":
        return {"y": la.decode_selective(*args, s["h"], **more), "h": s["h"]}
    if mode == "forward":
        y, h = la.forward_selective(*args, **more, h0=s["h0"], lens=s["lens"], out=s["out"], return_state=True)
        return {"y": y, "h": h}
    got = la.backward_selective(*args, s["dy"], **more, h0=s["h0"], dh=s["dh"])
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")
    return {n: v for n, v in zip(names, got) if v is not None}


def _own_conv(s):
    import kernelized_sequence_mixing_gb300 as la
    mode = s["case"]["mode"]
    if mode == "step":
        return {"y": la.decode_conv(s["x"], s["w"], s["state"], bias=s["bias"]), "state": s["state"]}
    if mode == "forward":
        y, state = la.forward_conv(s["x"], s["w"], bias=s["bias"], state=s["state"], lens=s["lens"], out=s["out"],
                                   return_state=True)
        return {"y": y, "state": state}
    got = la.backward_conv(s["x"], s["w"], s["dy"], bias=s["bias"], state=s["state"])
    return {n: v for n, v in zip(("dx", "dw", "dbias", "dstate"), got) if v is not None}


def _own_gate(s):
    import kernelized_sequence_mixing_gb300 as la
    case = s["case"]
    more = {"w": s["w"], "eps": EPS, "gate_first": case["gate_first"], "heads_first": case["heads_first"]}
    if case["mode"] == "forward":
        return la.forward_norm_gate(s["y"], s["gate"], **more)
    return dict(zip(("dy", "dgate", "dw"), la.backward_norm_gate(s["y"], s["gate"], s["do"], **more)))


def _own_residual(s):
    import kernelized_sequence_mixing_gb300 as la
    case = s["case"]
    if case["mode"] == "forward":
        return dict(zip(("o", "r"), la.forward_norm_residual(s["x"], s["residual"], w=s["w"], scale=case["scale"], eps=EPS)))
    got = la.backward_norm_residual(s["r"], s["do"], w=s["w"], dr=s["dr"], scale=case["scale"], eps=EPS)
    return dict(zip(("dresidual", "dx", "dw"), got))


OWN = {"selective": _own_selective, "conv": _own_conv, "norm_gate": _own_gate, "norm_residual": _own_residual}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# --------------------------------------------------------------------------- work

def work(case):
    """Bytes: every input read once and every output written once.  Flops: multiplications, additions and exponentials."""
    e = 4 if case["dtype"] == "float32" else 2
    op, mode = case["op"], case["mode"]
    if op == "norm_gate":
        n, p = case["B"] * case["H"] * case["L"] * case["D"], case["H"] * case["D"]
        return {"bytes": n * e * (3 if mode == "forward" else 5) + 4 * p * (1 if mode == "forward" else 2),
                "flops": n * (9 if mode == "forward" else 24)}
    if op == "norm_residual":
        n = case["R"] * case["E"]
        scaled = case["scale"] != 1.0  # dx and dresidual are one array otherwise
        return {"bytes": n * e * (4 if mode == "forward" else 4 + scaled) + 4 * case["E"] * (1 if mode == "forward" else 2),
                "flops": n * (6 if mode == "forward" else 12)}
    B, E = case["B"], case["E"]
    tokens = B if mode == "step" else sum(_lens(case))
    n = tokens * E
    if op == "conv":
        W = case["W"]
        params = 4 * E * (W + 1) * (2 if mode == "backward" else 1)
        state = B * (W - 1) * E * e * ((1 if mode == "forward" else 0) + (mode == "step" or case["start"]) * (1 if mode == "forward" else 2))
        return {"bytes": n * e * (3 if mode == "backward" else 2) + params + state, "flops": n * (2 * W + 5) * (3 if mode == "backward" else 1)}
    N, G, gate = case["N"], case["G"], case["gate"]
    params = 4 * (E * N + 2 * E) * (2 if mode == "backward" else 1)
    states = 4 * B * E * N * {"step": 2, "forward": 1 + case["start"], "backward": 3 * case["start"]}[mode]
    moved = (2 + 1 + gate) if mode != "backward" else (2 + gate + 1 + 2 + gate)
    shared = tokens * 2 * G * N * e * (2 if mode == "backward" else 1)
    return {"bytes": n * e * moved + shared + params + states, "flops": n * N * (7 if mode != "backward" else 24)}


# --------------------------------------------------------------------------- 64 bits

def _exact_selective(s):
    """The recurrence token by token; its gradients by automatic differentiation."""
    case = s["case"]
    back = case["mode"] == "backward"
    d = {k: v.double().requires_grad_(back and v.is_floating_point()) if torch.is_tensor(v) and k not in ("lens", "out", "dy", "dh") else v
         for k, v in s.items()}
    step = case["mode"] == "step"
    x, dt, z, Bm, Cm = ((v[:, None] if step and v is not None else v) for v in (d["x"], d["dt"], d["z"], d["Bm"], d["Cm"]))
    start = d["h"] if step else d["h0"]
    B, L, E, N, G = case["B"], x.shape[1], case["E"], case["N"], case["G"]
    h = start if start is not None else x.new_zeros(B, E, N)
    step_of = torch.logaddexp(dt + d["dt_bias"], torch.zeros_like(dt))
    lens = _lens(case) if not step else [1] * B
    live = torch.tensor(lens, device=x.device)
    ys = []
    for i in range(L):
        di, xi = step_of[:, i], x[:, i]
        b = Bm[:, i, :, None, :].expand(B, G, E // G, N).reshape(B, E, N)
        c = Cm[:, i, :, None, :].expand(B, G, E // G, N).reshape(B, E, N)
        new = torch.exp(di[..., None] * d["A"]) * h + (di * xi)[..., None] * b
        h = torch.where((i < live)[:, None, None], new, h) if case["ragged"] else new
        ys.append(torch.einsum("ben,ben->be", h, c) + d["D"] * xi)
    y = torch.stack(ys, 1)
    if z is not None:
        y = y * z / (1 + torch.exp(-z))
    if step:
        return {"y": y[:, 0], "h": h}
    if not back:
        if case["ragged"]:
            y = torch.where((torch.arange(L, device=x.device) < live[:, None])[..., None], y, s["out"].double())
        return {"y": y, "h": h}
    loss = (y * s["dy"].double()).sum()
    if s["dh"] is not None:
        loss = loss + (h * s["dh"].double()).sum()
    names = {"dx": "x", "ddt": "dt", "dA": "A", "dB": "Bm", "dC": "Cm", "dD": "D", "dz": "z", "ddt_bias": "dt_bias", "dh0": "h0"}
    names = {n: k for n, k in names.items() if d[k] is not None}
    return dict(zip(names, torch.autograd.grad(loss, [d[k] for k in names.values()])))


def _exact_conv(s):
    case = s["case"]
    step, back = case["mode"] == "step", case["mode"] == "backward"
    W = case["W"]
    x = (s["x"][:, None] if step else s["x"]).double()
    B, L, E = x.shape
    old = s["state"].double() if s["state"] is not None else x.new_zeros(B, W - 1, E)
    w, bias = s["w"].double(), s["bias"].double()
    leaves = [v.requires_grad_(back) for v in (x, w, bias, old)]
    rows = torch.cat((old, x), 1)
    y = torch.nn.functional.silu(torch.nn.functional.conv1d(rows.transpose(1, 2), w[:, None], bias, groups=E)).transpose(1, 2)
    if back:
        got = dict(zip(("dx", "dw", "dbias", "dstate"), torch.autograd.grad((y * s["dy"].double()).sum(), leaves)))
        if s["state"] is None:
            del got["dstate"]
        return got
    if step:
        return {"y": y[:, 0], "state": rows[:, 1:]}
    lens = _lens(case)
    y, state = y.clone(), []
    for b, n in enumerate(lens):
        if n < L:
            y[b, n:] = s["out"][b, n:].double()
        state.append(rows[b, n:n + W - 1])
    return {"y": y, "state": torch.stack(state)}


def _exact_gate(s):
    case = s["case"]
    y, gate, w = (s[k].double().requires_grad_(case["mode"] == "backward") for k in ("y", "gate", "w"))
    B, H, L, D = case["B"], case["H"], case["L"], case["D"]
    heads = torch.einsum("bhld->blhd", y) if case["heads_first"] else y
    act = torch.nn.functional.silu(gate).reshape(B, L, H, D)
    if case["gate_first"]:
        heads = heads * act
    o = heads / torch.sqrt(torch.linalg.vector_norm(heads, dim=-1, keepdim=True) ** 2 / D + EPS) * w
    if not case["gate_first"]:
        o = o * act
    o = o.reshape(B, L, H * D)
    if case["mode"] == "forward":
        return o
    return dict(zip(("dy", "dgate", "dw"), torch.autograd.grad((o * s["do"].double()).sum(), [y, gate, w])))


def _exact_residual(s):
    case = s["case"]
    w = s["w"].double().requires_grad_()
    if case["mode"] == "forward":
        r = torch.add(s["residual"].double(), s["x"].double(), alpha=case["scale"])
    else:
        r = s["r"].double().requires_grad_()
    o = w * r / torch.sqrt(torch.linalg.vector_norm(r, dim=-1, keepdim=True) ** 2 / r.shape[-1] + EPS)
    if case["mode"] == "forward":
        return {"o": o.detach(), "r": r}
    d, dw = torch.autograd.grad((o * s["do"].double()).sum() + (r * s["dr"].double()).sum(), [r, w])
    return {"dresidual": d, "dx": case["scale"] * d, "dw": dw}


EXACT = {"selective": _exact_selective, "conv": _exact_conv, "norm_gate": _exact_gate, "norm_residual": _exact_residual}


def exact(case, seed):
    # automatic differentiation keeps about eight 64-bit states a token
    if case["op"] == "selective" and case["mode"] == "backward" and case["L"] > 8192:
        return None
    return EXACT[case["op"]](prepare(case, seed))
