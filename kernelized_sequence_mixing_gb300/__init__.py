"""GB300 (sm_103a) kernelized linear attention, phi(x) = elu(x) + 1.

A thin ctypes binding over the C ABI in include/linattn.h (liblinattn.so,
built in-tree by ``kernelized_sequence_mixing_gb300.build``).  This module
only marshals arguments: shapes, dtypes, the current CUDA stream and, for host
tensors, the host<->device copies around the call.  Every step of the
computation runs in the library's CUDA kernels; there is no CPU fallback, and
a missing library raises RuntimeError.

Functions (same names as the C entry points, minus the ``la_`` prefix):
  forward(q, k, v, causal=True, gamma=None, eps=1e-6, out=None)
  prefill_state(k, v, gamma=None, S=None, z=None)
  decode_step(q, k, v, S, z, gamma=None, eps=1e-6, out=None)
  forward_state(q, k, v, gamma=None, eps=1e-6, out=None, S=None, z=None)
  forward_gated(q, k, v, a, eps=1e-6, out=None, return_state=False, S=None, z=None)
  decode_gated(q, k, v, a, S, z, eps=1e-6, out=None)
  favor_features(x, W, out=None)
  forward_favor(q, k, v, W, causal=True, gamma=None, eps=1e-6, out=None)
  backward(q, k, v, do, gamma=None, eps=1e-6)

The selective state space scan, its short convolution and the norms around a
block:
  forward_selective(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True,
                    h0=None, lens=None, out=None, return_state=False, h=None)
  decode_selective(x, dt, A, Bm, Cm, h, D=None, z=None, dt_bias=None, softplus=True, out=None)
  backward_selective(x, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, softplus=True,
                     h0=None, dh=None)
  forward_conv(x, w, bias=None, silu=True, state=None, lens=None, out=None,
               return_state=False, state_out=None)
  decode_conv(x, w, state, bias=None, silu=True, out=None)
  backward_conv(x, w, dy, bias=None, silu=True, state=None)
  forward_norm_gate(y, gate, w=None, eps=1e-5, gate_first=False, heads_first=True, out=None)
  backward_norm_gate(y, gate, do, w=None, eps=1e-5, gate_first=False, heads_first=True)
  forward_norm_residual(x, residual=None, w=None, scale=1.0, eps=1e-5, out=None, r=None)
  backward_norm_residual(r, do, w=None, dr=None, scale=1.0, eps=1e-5)
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from . import workloads  # noqa: F401  (seeded input generators)

__all__ = ["forward", "prefill_state", "decode_step", "forward_state",
           "forward_gated", "decode_gated", "favor_features", "forward_favor", "backward",
           "forward_selective", "decode_selective", "backward_selective",
           "forward_conv", "decode_conv", "backward_conv",
           "forward_norm_gate", "backward_norm_gate",
           "forward_norm_residual", "backward_norm_residual",
           "status_string",
           "device_wait_timeouts", "causal_kernel", "backward_kernel",
           "load_library", "library_path", "LinAttnError", "workloads"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "liblinattn.so")
_lib = None
_lock = threading.Lock()

LA_OK, LA_ERR_INVALID_ARG, LA_ERR_UNSUPPORTED, LA_ERR_CUDA = 0, 1, 2, 3
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


class LinAttnError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        super().__init__(f"{fn}: {status_string(code)} (status {code})")


def library_path() -> str:
    """Path of the in-tree liblinattn.so that load_library() opens."""
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load liblinattn.so; raises RuntimeError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"{_LIB_PATH} is missing: build it with "
                    "`python -m kernelized_sequence_mixing_gb300.build` "
                    "(or __graft_entry__.build()); there is no fallback path")
            lib = ctypes.CDLL(_LIB_PATH)
            P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
            FP = ctypes.POINTER(ctypes.c_float)
            lib.la_forward.argtypes = [P, P, P, P, I, I, I, I, I, I, FP, F, I, P]
            lib.la_forward_host.argtypes = [P, P, P, P, I, I, I, I, I, I, FP, F, I, P]
            lib.la_forward_host.restype = I
            lib.la_forward.restype = I
            lib.la_prefill_state.argtypes = [P, P, P, P, I, I, I, I, I, FP, I, P]
            lib.la_prefill_state.restype = I
            lib.la_forward_state.argtypes = [P, P, P, P, P, P, I, I, I, I, I, FP, F,
                                             I, P]
            lib.la_forward_state.restype = I
            lib.la_decode_step.argtypes = [P, P, P, P, P, P, I, I, I, I, FP, F,
                                           I, P]
            lib.la_decode_step.restype = I
            lib.la_forward_gated.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F,
                                             I, P]
            lib.la_forward_gated.restype = I
            lib.la_decode_gated.argtypes = [P, P, P, P, P, P, P, I, I, I, I, F, I, P]
            lib.la_decode_gated.restype = I
            lib.la_favor_features.argtypes = [P, P, P, I, I, I, I, P]
            lib.la_favor_features.restype = I
            lib.la_forward_favor.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, FP, F,
                                             I, P]
            lib.la_forward_favor.restype = I
            lib.la_backward.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, FP, F, I, P]
            lib.la_backward.restype = I
            lib.la_gated_kernel.argtypes = [I, I, I, I, I, I, I]
            lib.la_gated_kernel.restype = I
            lib.la_backward_launches.argtypes = [I, I, I, I, I, FP, I]
            lib.la_backward_launches.restype = I
            lib.la_backward_kernel.argtypes = [I, I, I, I, I, FP, I]
            lib.la_backward_kernel.restype = I
            lib.la_causal_kernel.argtypes = [I, I, I, I, I, FP, I]
            lib.la_causal_kernel.restype = I
            LL = ctypes.c_longlong
            lib.la_forward_selective.argtypes = [P] * 12 + [I] * 5 + [LL] * 5 + [I, I, P]
            lib.la_forward_selective.restype = I
            lib.la_decode_selective.argtypes = [P] * 10 + [I] * 4 + [LL] * 5 + [I, I, P]
            lib.la_decode_selective.restype = I
            lib.la_backward_selective.argtypes = [P] * 20 + [I] * 5 + [LL] * 5 + [I, I, P]
            lib.la_backward_selective.restype = I
            lib.la_forward_conv.argtypes = [P] * 7 + [I] * 4 + [LL, I, I, P]
            lib.la_forward_conv.restype = I
            lib.la_decode_conv.argtypes = [P] * 5 + [I] * 3 + [LL, I, I, P]
            lib.la_decode_conv.restype = I
            lib.la_backward_conv.argtypes = [P] * 9 + [I] * 4 + [LL, I, I, P]
            lib.la_backward_conv.restype = I
            lib.la_forward_norm_gate.argtypes = [P] * 4 + [I] * 6 + [F, I, P]
            lib.la_forward_norm_gate.restype = I
            lib.la_backward_norm_gate.argtypes = [P] * 7 + [I] * 6 + [F, I, P]
            lib.la_backward_norm_gate.restype = I
            lib.la_forward_norm_residual.argtypes = [P] * 5 + [LL, I, F, F, I, P]
            lib.la_forward_norm_residual.restype = I
            lib.la_backward_norm_residual.argtypes = [P] * 7 + [LL, I, F, F, I, P]
            lib.la_backward_norm_residual.restype = I
            lib.la_wait_selftest.argtypes = [ctypes.c_longlong, ctypes.POINTER(I)]
            lib.la_wait_selftest.restype = I
            lib.la_device_wait_timeouts.argtypes = [I]
            lib.la_device_wait_timeouts.restype = I
            lib.la_status_string.argtypes = [I]
            lib.la_status_string.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def status_string(code: int) -> str:
    """The library's text for a status code (la_status_string)."""
    return load_library().la_status_string(int(code)).decode()


def causal_kernel(B, H, N, D, Dv, gamma=None, dtype=torch.bfloat16) -> str:
    """Which kernel a causal forward with these sizes runs: "tensor-core-128"
    (128-token chunks), "tensor-core" (64-token chunks) or "cuda-core"
    (host-only query)."""
    code = load_library().la_causal_kernel(B, H, N, D, Dv, _gamma_arg(gamma, H),
                                           _DTYPES[dtype])
    if code < 0:
        raise LinAttnError("la_causal_kernel", -code)
    return {2: "tensor-core-128", 1: "tensor-core"}.get(code, "cuda-core")


def device_wait_timeouts(reset: bool = False) -> int:
    """Count of device-side bounded waits that gave up on the current device
    (nonzero: some kernel abandoned its work).  Synchronise first."""
    return int(load_library().la_device_wait_timeouts(1 if reset else 0))


def _gamma_arg(gamma, H):
    if gamma is None:
        return None
    if isinstance(gamma, torch.Tensor):
        vals = gamma.detach().to("cpu", torch.float32).reshape(-1).tolist()
    elif isinstance(gamma, (int, float)):
        vals = [float(gamma)] * H
    else:
        vals = [float(x) for x in gamma]
    if len(vals) != H:
        raise ValueError(f"gamma needs {H} values (one per head), got {len(vals)}")
    return (ctypes.c_float * H)(*vals)


def _dtype_code(t: torch.Tensor) -> int:
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}: use float32 or bfloat16")


def _stream(dev):
    index = torch.cuda.current_device() if dev.index is None else dev.index
    return torch._C._cuda_getCurrentRawStream(index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on(dev):
    """The context of a call on ``dev``: nothing to do where it is the current
    device already (the guard costs more than the rest of a short call)."""
    return _HERE if torch._C._cuda_getDevice() == dev.index else torch.cuda.device(dev)


_HERE = contextlib.nullcontext()


def _check(fn, code):
    if code != LA_OK:
        raise LinAttnError(fn, code)


def _contig(name, t):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# Device types whose memory the kernels may address.  The C entry points take
# plain pointers and cannot tell a host pointer or a short buffer from a good
# one, so every shape, dtype and device is checked here, before the call.
_DEVICE_TYPES = ("cuda",)


def _one_device(fn, named, allow_host=False):
    """All tensors of ``named`` [(name, tensor or None)] on one device, of a
    type the kernels can address (or the host, where ``allow_host``: the
    forward copies host tensors itself)."""
    dev = None
    for _, t in named:
        if t is not None:
            if dev is None:
                dev = t.device
                index = t.get_device()  # an integer: cheaper to compare; -1 is any other device
            elif t.get_device() != index or (index < 0 and t.device != dev):
                where = ", ".join(f"{n} on {t.device}" for n, t in named if t is not None)
                raise ValueError(f"{fn}: all tensors must be on one device ({where})")
    if dev.type not in _DEVICE_TYPES and not allow_host:
        raise ValueError(f"{fn}: tensors must be CUDA tensors, got {dev}")
    return dev


def _expect(fn, name, t, shape, dtype):
    """A caller-provided buffer: exactly ``shape`` and ``dtype``, contiguous."""
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{fn}: {name} must be {dtype}, got {t.dtype}")
    _contig(name, t)


def _qkv(fn, q, k, v, extra=()):
    """q, k: [B, H, N, D]; v: [B, H, N, Dv]; one dtype (plus ``extra`` named
    tensors of that dtype), contiguous.  Returns (B, H, N, D, Dv)."""
    for n, t in (("q", q), ("k", k), ("v", v)) + tuple(extra):
        _contig(n, t)
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError(f"{fn}: expected q, k: [B, H, N, D] and v: [B, H, N, Dv]")
    if not all(t.dtype == q.dtype for t in (k, v) + tuple(t for _, t in extra)):
        names = ", ".join(["q", "k", "v"] + [n for n, _ in extra])
        raise TypeError(f"{fn}: {names} must share one dtype")
    _dtype_code(q)
    B, H, N, D = q.shape
    return B, H, N, D, v.shape[-1]


def _step_qkv(fn, q, k, v):
    """Decode-step inputs q, k: [B, H, D]; v: [B, H, Dv]; one dtype."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _contig(n, t)
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[:2] != q.shape[:2]:
        raise ValueError(f"{fn}: expected q, k: [B, H, D] and v: [B, H, Dv]")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError(f"{fn}: q, k and v must share one dtype")
    _dtype_code(q)
    B, H, D = q.shape
    return B, H, D, v.shape[-1]


def forward(q, k, v, causal=True, gamma=None, eps=1e-6, out=None,
            device=None):
    """Linear attention over whole sequences.

    q, k: [B, H, N, D]; v: [B, H, N, Dv]; all float32 or all bfloat16,
    contiguous.  CUDA tensors are used in place on the current stream; host
    tensors go through la_forward_host on ``device`` (default cuda:0), which
    overlaps the copies with the kernels by groups of heads; the result is a
    host tensor (pinned), complete when this returns.  gamma: None, a float,
    or H per-head decays in [0, 1] (causal only).  Returns o: [B, H, N, Dv].
    """
    B, H, N, D, Dv = _qkv("forward", q, k, v)
    src = _one_device("forward", (("q", q), ("k", k), ("v", v), ("out", out)),
                      allow_host=True)
    if out is not None:
        _expect("forward", "out", out, (B, H, N, Dv), q.dtype)
    lib = load_library()
    host = src.type != "cuda"
    dev = torch.device(device or "cuda:0") if host else q.device
    dt = _dtype_code(q)
    g = _gamma_arg(gamma, H)
    with torch.cuda.device(dev):
        if host:
            qh, kh, vh = (t if t.is_pinned() else t.pin_memory() for t in (q, k, v))
            res = out if out is not None else torch.empty(
                (B, H, N, Dv), dtype=q.dtype, pin_memory=True)
            _check("la_forward_host", lib.la_forward_host(
                _ptr(qh), _ptr(kh), _ptr(vh), _ptr(res), B, H, N, D, Dv,
                1 if causal else 0, g, float(eps), dt, _stream(dev)))
            torch.cuda.current_stream(dev).synchronize()
            return res
        od = out if out is not None else torch.empty(
            (B, H, N, Dv), dtype=q.dtype, device=dev)
        _check("la_forward", lib.la_forward(
            _ptr(q), _ptr(k), _ptr(v), _ptr(od), B, H, N, D, Dv,
            1 if causal else 0, g, float(eps), dt, _stream(dev)))
        return od


def prefill_state(k, v, gamma=None, S=None, z=None):
    """State after a causal pass: S = sum_j gamma^(N-1-j) phi(k_j) v_j^T,
    z likewise.  k: [B, H, N, D], v: [B, H, N, Dv] CUDA tensors.  Returns
    (S [B, H, D, Dv] fp32, z [B, H, D] fp32), written into S, z if given."""
    _contig("k", k)
    _contig("v", v)
    if k.dim() != 4 or v.dim() != 4 or v.shape[:3] != k.shape[:3]:
        raise ValueError("prefill_state: expected k: [B, H, N, D] and v: [B, H, N, Dv]")
    if k.dtype != v.dtype:
        raise TypeError("prefill_state: k and v must share one dtype")
    _dtype_code(k)
    B, H, N, D = k.shape
    Dv = v.shape[-1]
    dev = _one_device("prefill_state", (("k", k), ("v", v), ("S", S), ("z", z)))
    if S is not None:
        _expect("prefill_state", "S", S, (B, H, D, Dv), torch.float32)
    if z is not None:
        _expect("prefill_state", "z", z, (B, H, D), torch.float32)
    lib = load_library()
    with torch.cuda.device(dev):
        if S is None:
            S = torch.empty((B, H, D, Dv), dtype=torch.float32, device=dev)
        if z is None:
            z = torch.empty((B, H, D), dtype=torch.float32, device=dev)
        _check("la_prefill_state", lib.la_prefill_state(
            _ptr(k), _ptr(v), _ptr(S), _ptr(z), B, H, N, D, Dv,
            _gamma_arg(gamma, H), _dtype_code(k), _stream(dev)))
    return S, z


def forward_state(q, k, v, gamma=None, eps=1e-6, out=None, S=None, z=None):
    """Causal forward that also returns the state after the last token:
    (o [B, H, N, Dv], S [B, H, D, Dv] fp32, z [B, H, D] fp32), the state the
    decode loop continues from.  q, k: [B, H, N, D]; v: [B, H, N, Dv] CUDA
    tensors of one dtype; out, S, z: optional destinations."""
    fn = "forward_state"
    B, H, N, D, Dv = _qkv(fn, q, k, v)
    dev = _one_device(fn, (("q", q), ("k", k), ("v", v), ("out", out), ("S", S), ("z", z)))
    if out is not None:
        _expect(fn, "out", out, (B, H, N, Dv), q.dtype)
    if S is not None:
        _expect(fn, "S", S, (B, H, D, Dv), torch.float32)
    if z is not None:
        _expect(fn, "z", z, (B, H, D), torch.float32)
    lib = load_library()
    with torch.cuda.device(dev):
        o = out if out is not None else torch.empty((B, H, N, Dv), dtype=q.dtype, device=dev)
        if S is None:
            S = torch.empty((B, H, D, Dv), dtype=torch.float32, device=dev)
        if z is None:
            z = torch.empty((B, H, D), dtype=torch.float32, device=dev)
        _check("la_forward_state", lib.la_forward_state(
            _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(S), _ptr(z), B, H, N, D, Dv,
            _gamma_arg(gamma, H), float(eps), _dtype_code(q), _stream(dev)))
    return o, S, z


def decode_step(q, k, v, S, z, gamma=None, eps=1e-6, out=None):
    """One recurrent step in place on (S, z): update with (k, v), then read
    out with q.  q, k: [B, H, D]; v: [B, H, Dv]; S: [B, H, D, Dv] fp32;
    z: [B, H, D] fp32 (all CUDA).  Returns o: [B, H, Dv]."""
    fn = "decode_step"
    B, H, D, Dv = _step_qkv(fn, q, k, v)
    dev = _one_device(fn, (("q", q), ("k", k), ("v", v), ("S", S), ("z", z), ("out", out)))
    _expect(fn, "S", S, (B, H, D, Dv), torch.float32)
    _expect(fn, "z", z, (B, H, D), torch.float32)
    if out is not None:
        _expect(fn, "out", out, (B, H, Dv), q.dtype)
    lib = load_library()
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty((B, H, Dv), dtype=q.dtype, device=dev)
        _check("la_decode_step", lib.la_decode_step(
            _ptr(q), _ptr(k), _ptr(v), _ptr(S), _ptr(z), _ptr(out), B, H, D,
            Dv, _gamma_arg(gamma, H), float(eps), _dtype_code(q),
            _stream(dev)))
    return out


def forward_gated(q, k, v, a, eps=1e-6, out=None, return_state=False, S=None, z=None):
    """Gated causal forward: S_t = diag(a_t) S_(t-1) + phi(k_t) v_t^T,
    z_t = a_t * z_(t-1) + phi(k_t), o_t = phi(q_t)^T S_t / (phi(q_t).z_t + eps).
    q, k: [B, H, N, D]; v: [B, H, N, Dv] CUDA tensors of one dtype; a:
    [B, H, N, D] float32 gates in [0, 1] on the same device.  Returns o, or
    (o, S [B, H, D, Dv] fp32, z [B, H, D] fp32) with the state after the last
    token when return_state is true (or S, z are given)."""
    fn = "forward_gated"
    B, H, N, D, Dv = _qkv(fn, q, k, v)
    _expect(fn, "a", a, (B, H, N, D), torch.float32)
    dev = _one_device(fn, (("q", q), ("k", k), ("v", v), ("a", a), ("out", out), ("S", S),
                           ("z", z)))
    if out is not None:
        _expect(fn, "out", out, (B, H, N, Dv), q.dtype)
    if S is not None:
        _expect(fn, "S", S, (B, H, D, Dv), torch.float32)
    if z is not None:
        _expect(fn, "z", z, (B, H, D), torch.float32)
    lib = load_library()
    want_state = return_state or S is not None or z is not None
    with torch.cuda.device(dev):
        o = out if out is not None else torch.empty((B, H, N, Dv), dtype=q.dtype, device=dev)
        if want_state:
            if S is None:
                S = torch.empty((B, H, D, Dv), dtype=torch.float32, device=dev)
            if z is None:
                z = torch.empty((B, H, D), dtype=torch.float32, device=dev)
        _check("la_forward_gated", lib.la_forward_gated(
            _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(o),
            _ptr(S) if want_state else None, _ptr(z) if want_state else None,
            B, H, N, D, Dv, float(eps), _dtype_code(q), _stream(dev)))
    return (o, S, z) if want_state else o


def decode_gated(q, k, v, a, S, z, eps=1e-6, out=None):
    """One gated recurrent step in place on (S, z): S <- diag(a) S +
    phi(k) v^T, z <- a * z + phi(k), then read out with q.  q, k, a: [B, H, D]
    (a float32); v: [B, H, Dv]; S: [B, H, D, Dv] fp32; z: [B, H, D] fp32 (all
    CUDA).  Returns o: [B, H, Dv]."""
    fn = "decode_gated"
    B, H, D, Dv = _step_qkv(fn, q, k, v)
    dev = _one_device(fn, (("q", q), ("k", k), ("v", v), ("a", a), ("S", S), ("z", z),
                           ("out", out)))
    _expect(fn, "a", a, (B, H, D), torch.float32)
    _expect(fn, "S", S, (B, H, D, Dv), torch.float32)
    _expect(fn, "z", z, (B, H, D), torch.float32)
    if out is not None:
        _expect(fn, "out", out, (B, H, Dv), q.dtype)
    lib = load_library()
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty((B, H, Dv), dtype=q.dtype, device=dev)
        _check("la_decode_gated", lib.la_decode_gated(
            _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(S), _ptr(z), _ptr(out), B, H, D,
            Dv, float(eps), _dtype_code(q), _stream(dev)))
    return out


def favor_features(x, W, out=None):
    """Performer random features phi(x) = r^(-1/2) exp(W x - |x|^2 / 2) of
    every row of x [..., D] with the directions W [r, D] (same dtype, CUDA).
    Returns [..., r]."""
    fn = "favor_features"
    _contig("x", x)
    _contig("W", W)
    if x.dim() < 1 or W.dim() != 2 or W.shape[1] != x.shape[-1]:
        raise ValueError(f"{fn}: W must be [r, D] for x [..., D]")
    if W.dtype != x.dtype:
        raise TypeError(f"{fn}: W must have the dtype of x")
    _dtype_code(x)
    D, r = x.shape[-1], W.shape[0]
    rows = x.numel() // D if D else 0
    dev = _one_device(fn, (("x", x), ("W", W), ("out", out)))
    if out is not None:
        _expect(fn, "out", out, tuple(x.shape[:-1]) + (r,), x.dtype)
    lib = load_library()
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty(x.shape[:-1] + (r,), dtype=x.dtype, device=dev)
        _check("la_favor_features", lib.la_favor_features(
            _ptr(x), _ptr(W), _ptr(out), rows, D, r, _dtype_code(x), _stream(dev)))
    return out


def forward_favor(q, k, v, W, causal=True, gamma=None, eps=1e-6, out=None):
    """Performer attention: the random features of q and k with the
    directions W [r, D], then linear attention over them (causal with
    optional per-head decay, or non-causal).  q, k: [B, H, N, D]; v:
    [B, H, N, Dv]; all CUDA tensors of one dtype.  Returns o [B, H, N, Dv]."""
    fn = "forward_favor"
    B, H, N, D, Dv = _qkv(fn, q, k, v, extra=(("W", W),))
    if W.dim() != 2 or W.shape[1] != D:
        raise ValueError(f"{fn}: W must be [r, D]")
    r = W.shape[0]
    dev = _one_device(fn, (("q", q), ("k", k), ("v", v), ("W", W), ("out", out)))
    if out is not None:
        _expect(fn, "out", out, (B, H, N, Dv), q.dtype)
    lib = load_library()
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty((B, H, N, Dv), dtype=q.dtype, device=dev)
        _check("la_forward_favor", lib.la_forward_favor(
            _ptr(q), _ptr(k), _ptr(v), _ptr(W), _ptr(out), B, H, N, D, Dv, r,
            1 if causal else 0, _gamma_arg(gamma, H), float(eps), _dtype_code(q),
            _stream(dev)))
    return out


def backward(q, k, v, do, gamma=None, eps=1e-6, dq=None, dk=None, dv=None):
    """Gradients (dq, dk, dv) of the causal forward o = forward(q, k, v,
    causal=True, gamma, eps) for the upstream gradient do = dL/do.  q, k:
    [B, H, N, D]; v, do: [B, H, N, Dv]; CUDA tensors of one dtype."""
    fn = "backward"
    B, H, N, D, Dv = _qkv(fn, q, k, v, extra=(("do", do),))
    if do.shape != v.shape:
        raise ValueError(f"{fn}: do must have the shape of v")
    dev = _one_device(fn, (("q", q), ("k", k), ("v", v), ("do", do), ("dq", dq), ("dk", dk),
                           ("dv", dv)))
    for n, t, shape in (("dq", dq, q.shape), ("dk", dk, k.shape), ("dv", dv, v.shape)):
        if t is not None:
            _expect(fn, n, t, shape, q.dtype)
    lib = load_library()
    with torch.cuda.device(dev):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        _check("la_backward", lib.la_backward(
            _ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, D, Dv,
            _gamma_arg(gamma, H), float(eps), _dtype_code(q), _stream(dev)))
    return dq, dk, dv


def backward_launches(B, H, N, D, Dv, gamma=None, dtype=torch.bfloat16) -> int:
    """Kernels one backward() call with these arguments launches on the
    current device."""
    n = load_library().la_backward_launches(B, H, N, D, Dv, _gamma_arg(gamma, H), _DTYPES[dtype])
    if n < 0:
        raise LinAttnError("la_backward_launches", -n)
    return int(n)


def backward_kernel(B, H, N, D, Dv, gamma=None, dtype=torch.bfloat16) -> str:
    """Which kernels backward() runs: "tensor-core" (bf16, Dv = 64, every
    decay >= 0.35) or "cuda-core".  Host-only query."""
    code = load_library().la_backward_kernel(B, H, N, D, Dv, _gamma_arg(gamma, H), _DTYPES[dtype])
    if code < 0:
        raise LinAttnError("la_backward_kernel", -code)
    return "tensor-core" if code == 1 else "cuda-core"


def gated_kernel(B, H, N, D, Dv, dtype=torch.bfloat16, want_state=False) -> str:
    """Which form forward_gated runs: "tensor-core" (it still falls back to
    the CUDA-core form at run time when some chunk's gates forget harder
    than 2^-93) or "cuda-core"; the final state does not change the choice.
    Host-only query."""
    code = load_library().la_gated_kernel(B, H, N, D, Dv, _DTYPES[dtype], 1 if want_state else 0)
    if code < 0:
        raise LinAttnError("la_gated_kernel", -code)
    return "tensor-core" if code == 1 else "cuda-core"


def wait_selftest(cycles=2_000_000) -> bool:
    """Run the kernels' bounded wait on a barrier nothing arrives on, with a
    short limit: True if it gave up (and counted itself in
    device_wait_timeouts), as it should.  Synchronises the device."""
    gave_up = ctypes.c_int(0)
    _check("la_wait_selftest", load_library().la_wait_selftest(int(cycles), ctypes.byref(gave_up)))
    return bool(gave_up.value)


# --- selective state space scan, short convolution, norms around a block ---


def _c_ints(fn, *sizes):
    """Sizes that reach the library as C ints, which ctypes cuts to 32 bits
    without a word."""
    if max(sizes) > 0x7fffffff:
        raise ValueError(f"{fn}: sizes of 2^31 and more are not supported (got {sizes})")


def _tokens(fn, name, t, lead, row, dtype):
    """The token stride (0: dense) of an input [*lead, *row] of ``dtype`` whose
    rows are contiguous; lead is (B, L), with L token strides between
    sequences, or (B,): dense tensors and slices of a dense tensor's rows."""
    if t.shape != lead + row:
        raise ValueError(f"{fn}: {name} must have shape {lead + row}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{fn}: {name} must be {dtype}, got {t.dtype}")
    if t.is_contiguous():
        return 0
    stride = t.stride()
    width = 1
    for size, st in zip(reversed(row), reversed(stride)):
        if size > 1 and st != width:
            raise ValueError(f"{fn}: the values of each token of {name} must be contiguous")
        width *= size
    ld = width
    for i in range(len(lead) - 1, -1, -1):
        if lead[i] > 1:
            ld = stride[i]
            break
    if ld < width or ld % 8 or (len(lead) == 2 and lead[0] > 1 and lead[1] > 1
                                and stride[0] != lead[1] * ld):
        raise ValueError(f"{fn}: {name} must be dense or a slice of a dense tensor's rows, with a "
                         f"multiple of 8 elements between tokens (strides {stride})")
    return ld


def _param(fn, name, t, shape):
    """An optional fp32 parameter or state: exactly ``shape``, contiguous."""
    if t is not None:
        _expect(fn, name, t, shape, torch.float32)


def _scan_args(fn, x, dt, A, Bm, Cm, D, z, dt_bias, dims):
    """Checks shared by the scan's entry points; ``dims`` is 3 for sequences,
    2 for one token.  Returns (lead, E, N, G, token strides)."""
    if x.dim() != dims or Bm.dim() != dims + 1 or A.dim() != 2:
        tok = "B, L" if dims == 3 else "B"
        raise ValueError(f"{fn}: expected x, dt: [{tok}, E], A: [E, N] and Bm, Cm: [{tok}, G, N]")
    dtype = x.dtype
    if dtype not in _DTYPES:
        _dtype_code(x)
    *lead, E = x.shape
    lead = tuple(lead)
    G, N = Bm.shape[-2:]
    _c_ints(fn, *lead, E, G, N)
    tok, grp = lead + (E,), lead + (G, N)
    lds = []
    for name, t, shape in (("x", x, tok), ("dt", dt, tok), ("z", z, tok), ("Bm", Bm, grp), ("Cm", Cm, grp)):
        # dense rows need no stride; _tokens finds the others' and every fault
        lds.append(0 if t is None or (t.shape == shape and t.dtype is dtype and t.is_contiguous())
                   else _tokens(fn, name, t, lead, shape[len(lead):], dtype))
    _param(fn, "A", A, (E, N))
    _param(fn, "D", D, (E,))
    _param(fn, "dt_bias", dt_bias, (E,))
    return lead, E, N, G, lds


def _lens(fn, lens, B):
    if lens is not None:
        _expect(fn, "lens", lens, (B,), torch.int32)


def forward_selective(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True, h0=None,
                      lens=None, out=None, return_state=False, h=None):
    """Selective state space scan: dt_t = softplus(dt_t + dt_bias) (or the
    sum), h_t = exp(dt_t A) h_(t-1) + dt_t x_t B_t, y_t = (C_t . h_t + D x_t)
    silu(z_t).  x, dt, z: [B, L, E]; Bm, Cm: [B, L, G, N] CUDA tensors of one
    dtype, dense or slices of a dense tensor's rows; A: [E, N], D, dt_bias: [E]
    and h0: [B, E, N] float32; lens: [B] int32 tokens per sequence (rows behind
    have no effect and stay unwritten).  States are meant to decay (steps times A
    not positive).  Returns y, or (y, h [B, E, N] float32) with
    the state after the last token when return_state is true (or h is given)."""
    fn = "forward_selective"
    (B, L), E, N, G, lds = _scan_args(fn, x, dt, A, Bm, Cm, D, z, dt_bias, 3)
    _param(fn, "h0", h0, (B, E, N))
    _param(fn, "h", h, (B, E, N))
    _lens(fn, lens, B)
    if out is not None:
        _expect(fn, "out", out, (B, L, E), x.dtype)
    dev = _one_device(fn, (("x", x), ("dt", dt), ("A", A), ("Bm", Bm), ("Cm", Cm), ("D", D),
                           ("z", z), ("dt_bias", dt_bias), ("h0", h0), ("lens", lens),
                           ("out", out), ("h", h)))
    lib = load_library()
    with _on(dev):
        if out is None:
            out = torch.empty((B, L, E), dtype=x.dtype, device=dev)
        if h is None and return_state:
            h = torch.empty((B, E, N), dtype=torch.float32, device=dev)
        _check("la_forward_selective", lib.la_forward_selective(
            _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z), _ptr(dt_bias),
            _ptr(h0), _ptr(lens), _ptr(out), _ptr(h), B, L, E, N, G, *lds,
            1 if softplus else 0, _DTYPES[x.dtype], _stream(dev)))
    return out if h is None else (out, h)


def decode_selective(x, dt, A, Bm, Cm, h, D=None, z=None, dt_bias=None, softplus=True, out=None):
    """One token of the scan, in place on h [B, E, N] float32.  x, dt, z:
    [B, E]; Bm, Cm: [B, G, N]; otherwise as forward_selective.  Returns
    y: [B, E]."""
    fn = "decode_selective"
    (B,), E, N, G, lds = _scan_args(fn, x, dt, A, Bm, Cm, D, z, dt_bias, 2)
    _expect(fn, "h", h, (B, E, N), torch.float32)
    if out is not None:
        _expect(fn, "out", out, (B, E), x.dtype)
    dev = _one_device(fn, (("x", x), ("dt", dt), ("A", A), ("Bm", Bm), ("Cm", Cm), ("h", h),
                           ("D", D), ("z", z), ("dt_bias", dt_bias), ("out", out)))
    lib = load_library()
    with _on(dev):
        if out is None:
            out = torch.empty((B, E), dtype=x.dtype, device=dev)
        _check("la_decode_selective", lib.la_decode_selective(
            _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z), _ptr(dt_bias),
            _ptr(h), _ptr(out), B, E, N, G, *lds, 1 if softplus else 0, _DTYPES[x.dtype],
            _stream(dev)))
    return out


def backward_selective(x, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, softplus=True,
                       h0=None, dh=None):
    """Gradients of y (and the final state) = forward_selective(...) for the
    upstream gradients dy [B, L, E] of y and, if given, dh [B, E, N] float32
    of the final state.  Returns (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0);
    dD, dz, ddt_bias and dh0 are None where their input is.  A batch padded at
    the end takes zero rows of dy and finite padding, with dh also steps of zero
    there (raw dt -inf under softplus)."""
    fn = "backward_selective"
    (B, L), E, N, G, lds = _scan_args(fn, x, dt, A, Bm, Cm, D, z, dt_bias, 3)
    _expect(fn, "dy", dy, (B, L, E), x.dtype)
    _param(fn, "h0", h0, (B, E, N))
    _param(fn, "dh", dh, (B, E, N))
    dev = _one_device(fn, (("x", x), ("dt", dt), ("A", A), ("Bm", Bm), ("Cm", Cm), ("dy", dy),
                           ("D", D), ("z", z), ("dt_bias", dt_bias), ("h0", h0), ("dh", dh)))
    lib = load_library()
    f = torch.float32
    with _on(dev):
        new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        dx, ddt = new((B, L, E), x.dtype), new((B, L, E), x.dtype)
        dA, dB, dC = new((E, N), f), new((B, L, G, N), x.dtype), new((B, L, G, N), x.dtype)
        dD = new((E,), f) if D is not None else None
        dz = new((B, L, E), x.dtype) if z is not None else None
        dbias = new((E,), f) if dt_bias is not None else None
        dh0 = new((B, E, N), f) if h0 is not None else None
        _check("la_backward_selective", lib.la_backward_selective(
            _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z), _ptr(dt_bias),
            _ptr(h0), _ptr(dy), _ptr(dh), _ptr(dx), _ptr(ddt), _ptr(dA), _ptr(dB), _ptr(dC),
            _ptr(dD), _ptr(dz), _ptr(dbias), _ptr(dh0), B, L, E, N, G, *lds,
            1 if softplus else 0, _DTYPES[x.dtype], _stream(dev)))
    return dx, ddt, dA, dB, dC, dD, dz, dbias, dh0


def _conv_args(fn, x, w, bias, dims):
    if x.dim() != dims or w.dim() != 2:
        raise ValueError(f"{fn}: expected x: [{'B, L' if dims == 3 else 'B'}, E] and w: [E, W]")
    _dtype_code(x)
    lead, E = tuple(x.shape[:-1]), x.shape[-1]
    W = w.shape[1]
    _c_ints(fn, *lead, E, W)
    _param(fn, "w", w, (E, W))
    _param(fn, "bias", bias, (E,))
    return lead, E, W, _tokens(fn, "x", x, lead, (E,), x.dtype)


def forward_conv(x, w, bias=None, silu=True, state=None, lens=None, out=None,
                 return_state=False, state_out=None):
    """Short causal depthwise convolution: y_t = act(bias + sum_k w[:, k]
    x_(t - W + 1 + k)), act = SiLU (or none).  x: [B, L, E] (dense, or a slice
    of a dense tensor's rows), w: [E, W] float32 with W in 2..4, bias: [E]
    float32, state: [B, W - 1, E] of x's dtype, the rows before the first
    token (zeros without it), lens: [B] int32 tokens per sequence.  Returns y,
    or (y, state after the last token) when return_state is true (or state_out
    is given)."""
    fn = "forward_conv"
    (B, L), E, W, ld = _conv_args(fn, x, w, bias, 3)
    for n, t in (("state", state), ("state_out", state_out)):
        if t is not None:
            _expect(fn, n, t, (B, W - 1, E), x.dtype)
    _lens(fn, lens, B)
    if out is not None:
        _expect(fn, "out", out, (B, L, E), x.dtype)
    dev = _one_device(fn, (("x", x), ("w", w), ("bias", bias), ("state", state), ("lens", lens),
                           ("out", out), ("state_out", state_out)))
    lib = load_library()
    with _on(dev):
        if out is None:
            out = torch.empty((B, L, E), dtype=x.dtype, device=dev)
        if state_out is None and return_state:
            state_out = torch.empty((B, max(W - 1, 0), E), dtype=x.dtype, device=dev)
        _check("la_forward_conv", lib.la_forward_conv(
            _ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(lens), _ptr(out), _ptr(state_out),
            B, L, E, W, ld, 1 if silu else 0, _DTYPES[x.dtype], _stream(dev)))
    return out if state_out is None else (out, state_out)


def decode_conv(x, w, state, bias=None, silu=True, out=None):
    """One token of the convolution, in place on state [B, W - 1, E]: x [B, E].
    Returns y: [B, E]."""
    fn = "decode_conv"
    (B,), E, W, ld = _conv_args(fn, x, w, bias, 2)
    _expect(fn, "state", state, (B, W - 1, E), x.dtype)
    if out is not None:
        _expect(fn, "out", out, (B, E), x.dtype)
    dev = _one_device(fn, (("x", x), ("w", w), ("state", state), ("bias", bias), ("out", out)))
    lib = load_library()
    with _on(dev):
        if out is None:
            out = torch.empty((B, E), dtype=x.dtype, device=dev)
        _check("la_decode_conv", lib.la_decode_conv(
            _ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(out), B, E, W, ld,
            1 if silu else 0, _DTYPES[x.dtype], _stream(dev)))
    return out


def backward_conv(x, w, dy, bias=None, silu=True, state=None):
    """Gradients (dx, dw, dbias, dstate) of forward_conv(x, w, bias, silu,
    state) for the upstream gradient dy [B, L, E]; dbias and dstate are None
    where their input is.  A batch padded at the end takes zero rows of dy and
    finite rows of x there."""
    fn = "backward_conv"
    (B, L), E, W, ld = _conv_args(fn, x, w, bias, 3)
    _expect(fn, "dy", dy, (B, L, E), x.dtype)
    if state is not None:
        _expect(fn, "state", state, (B, W - 1, E), x.dtype)
    dev = _one_device(fn, (("x", x), ("w", w), ("dy", dy), ("bias", bias), ("state", state)))
    lib = load_library()
    with _on(dev):
        dx = torch.empty((B, L, E), dtype=x.dtype, device=dev)
        dw = torch.empty((E, W), dtype=torch.float32, device=dev)
        dbias = torch.empty((E,), dtype=torch.float32, device=dev) if bias is not None else None
        dstate = torch.empty_like(state) if state is not None else None
        _check("la_backward_conv", lib.la_backward_conv(
            _ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(dy), _ptr(dx), _ptr(dw), _ptr(dbias),
            _ptr(dstate), B, L, E, W, ld, 1 if silu else 0, _DTYPES[x.dtype], _stream(dev)))
    return dx, dw, dbias, dstate


def _norm_gate_args(fn, y, gate, w, heads_first, extra=()):
    if y.dim() != 4:
        raise ValueError(f"{fn}: expected y: [B, H, L, D] (heads_first) or [B, L, H, D]")
    _contig("y", y)
    _dtype_code(y)
    B, H, L, D = y.shape
    if not heads_first:
        H, L = L, H
    _c_ints(fn, B, H, L, D)
    for n, t in (("gate", gate),) + tuple(extra):
        if t is not None:
            _expect(fn, n, t, (B, L, H * D), y.dtype)
    _param(fn, "w", w, (H, D))
    return B, H, L, D


def forward_norm_gate(y, gate, w=None, eps=1e-5, gate_first=False, heads_first=True, out=None):
    """RMS norm of each head's rows with a SiLU gate: norm(y) w silu(gate), or
    norm(y silu(gate)) w when gate_first.  y: [B, H, L, D] as forward() returns
    it, or [B, L, H, D] with heads_first=False; gate: [B, L, H*D]; one dtype,
    contiguous; w: [H, D] float32.  Returns o: [B, L, H*D]."""
    fn = "forward_norm_gate"
    B, H, L, D = _norm_gate_args(fn, y, gate, w, heads_first, (("out", out),))
    dev = _one_device(fn, (("y", y), ("gate", gate), ("w", w), ("out", out)))
    lib = load_library()
    with _on(dev):
        if out is None:
            out = torch.empty((B, L, H * D), dtype=y.dtype, device=dev)
        _check("la_forward_norm_gate", lib.la_forward_norm_gate(
            _ptr(y), _ptr(gate), _ptr(w), _ptr(out), B, H, L, D, 1 if heads_first else 0,
            1 if gate_first else 0, float(eps), _DTYPES[y.dtype], _stream(dev)))
    return out


def backward_norm_gate(y, gate, do, w=None, eps=1e-5, gate_first=False, heads_first=True):
    """Gradients (dy, dgate, dw) of forward_norm_gate for the upstream gradient
    do [B, L, H*D]; dy is laid out as y, dw is None without w."""
    fn = "backward_norm_gate"
    B, H, L, D = _norm_gate_args(fn, y, gate, w, heads_first, (("do", do),))
    dev = _one_device(fn, (("y", y), ("gate", gate), ("do", do), ("w", w)))
    lib = load_library()
    with _on(dev):
        dy, dgate = torch.empty_like(y), torch.empty_like(gate)
        dw = torch.empty((H, D), dtype=torch.float32, device=dev) if w is not None else None
        _check("la_backward_norm_gate", lib.la_backward_norm_gate(
            _ptr(y), _ptr(gate), _ptr(w), _ptr(do), _ptr(dy), _ptr(dgate), _ptr(dw), B, H, L, D,
            1 if heads_first else 0, 1 if gate_first else 0, float(eps), _DTYPES[y.dtype],
            _stream(dev)))
    return dy, dgate, dw


def _rows(fn, name, t, others, w):
    """Rows [..., E] of one dtype and shape; returns (rows, E)."""
    if t.dim() < 1:
        raise ValueError(f"{fn}: expected {name}: [..., E]")
    _contig(name, t)
    _dtype_code(t)
    for n, o in others:
        if o is not None:
            _expect(fn, n, o, t.shape, t.dtype)
    E = t.shape[-1]
    _c_ints(fn, E)
    _param(fn, "w", w, (E,))
    return (t.numel() // E if E else 0), E


def forward_norm_residual(x, residual=None, w=None, scale=1.0, eps=1e-5, out=None, r=None):
    """r = residual + scale x (scale x without a residual) and its RMS norm
    o = r rsqrt(mean r^2 + eps) w over the last dimension.  x, residual:
    [..., E] of one dtype; w: [E] float32.  Returns (o, r)."""
    fn = "forward_norm_residual"
    rows, E = _rows(fn, "x", x, (("residual", residual), ("out", out), ("r", r)), w)
    dev = _one_device(fn, (("x", x), ("residual", residual), ("w", w), ("out", out), ("r", r)))
    lib = load_library()
    with _on(dev):
        if out is None:
            out = torch.empty_like(x)
        if r is None:
            r = torch.empty_like(x)
        _check("la_forward_norm_residual", lib.la_forward_norm_residual(
            _ptr(x), _ptr(residual), _ptr(w), _ptr(out), _ptr(r), rows, E, float(scale),
            float(eps), _DTYPES[x.dtype], _stream(dev)))
    return out, r


def backward_norm_residual(r, do, w=None, dr=None, scale=1.0, eps=1e-5):
    """Gradients (dresidual, dx, dw) of forward_norm_residual at its r, for the
    upstream gradients do of o and dr of r (None: none).  With scale = 1 dx is
    dresidual itself; dw is None without w."""
    fn = "backward_norm_residual"
    rows, E = _rows(fn, "r", r, (("do", do), ("dr", dr)), w)
    dev = _one_device(fn, (("r", r), ("do", do), ("dr", dr), ("w", w)))
    lib = load_library()
    with _on(dev):
        dres = torch.empty_like(r)
        dx = torch.empty_like(r) if scale != 1.0 else None
        dw = torch.empty((E,), dtype=torch.float32, device=dev) if w is not None else None
        _check("la_backward_norm_residual", lib.la_backward_norm_residual(
            _ptr(r), _ptr(w), _ptr(do), _ptr(dr), _ptr(dres), _ptr(dx), _ptr(dw), rows, E,
            float(scale), float(eps), _DTYPES[r.dtype], _stream(dev)))
    return dres, (dres if dx is None else dx), dw
