"""ctypes binding of libla_b200.so (include/la.h), one Python function per
C entry point, with the same names.

Argument marshalling only: shapes become an ``la_desc``, tensors become their
device pointers, the stream is torch's current CUDA stream unless one is
given. All computation happens in the library's CUDA kernels; if the library
cannot be loaded, every call raises (there is no fallback).

Tensors are contiguous [B, H, N, d] (q, k, v, out; float32 or bfloat16),
S [B, H, d, d] and z [B, H, d] float32, m [B, N] int32. ``phi`` is "relu1"
(relu(x)+1) or "identity".
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libla_b200.so")

LA_OK = 0
STATUS_NAMES = {0: "LA_OK", 1: "LA_ERR_INVALID_ARG", 2: "LA_ERR_UNSUPPORTED",
                3: "LA_ERR_MISALIGNED", 4: "LA_ERR_WORKSPACE", 5: "LA_ERR_CUDA",
                6: "LA_ERR_MASK_RANGE", 7: "LA_ERR_TIMEOUT"}
DTYPES = {torch.float32: 0, torch.bfloat16: 1}
PHIS = {"relu1": 0, "identity": 1, "elu1": 2}
OPS = {"kv_summary": 0, "noncausal": 1, "causal": 2, "prefix": 3, "decode": 4, "noncausal_bwd": 5,
       "causal_bwd": 6, "gated_causal": 8, "gated_causal_bwd": 9}


class LaError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")


class la_desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("phi", ctypes.c_int32),
                ("normalize", ctypes.c_int32)]


class la_rope_desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hk", ctypes.c_int32),
                ("d", ctypes.c_int32), ("rot", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("table_rows", ctypes.c_int32), ("eps", ctypes.c_float)]


class la_strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("n", ctypes.c_int64), ("h", ctypes.c_int64)]


_lib = None

_P = ctypes.c_void_p
_ROPE = [ctypes.POINTER(la_rope_desc), _P, ctypes.POINTER(la_strides), _P, ctypes.POINTER(la_strides), _P, _P, _P, _P, _P]
_SIGS = {
    "la_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(la_desc), ctypes.c_int32, ctypes.c_int32]),
    "la_kv_summary": (ctypes.c_int, [ctypes.POINTER(la_desc), _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "la_noncausal": (ctypes.c_int, [ctypes.POINTER(la_desc), _P, _P, _P, _P, _P, _P, _P,
                                    ctypes.c_size_t, _P]),
    "la_causal_chunked": (ctypes.c_int, [ctypes.POINTER(la_desc), ctypes.c_int32, _P, _P, _P, _P,
                                         _P, ctypes.c_size_t, _P]),
    "la_causal_prefill": (ctypes.c_int, [ctypes.POINTER(la_desc), ctypes.c_int32, _P, _P, _P, _P, _P, _P,
                                         _P, ctypes.c_size_t, _P]),
    "la_noncausal_backward": (ctypes.c_int, [ctypes.POINTER(la_desc), _P, _P, _P, _P, _P, _P, _P, _P,
                                             ctypes.c_size_t, _P]),
    "la_causal_backward": (ctypes.c_int, [ctypes.POINTER(la_desc), _P, _P, _P, _P, _P, _P, _P, _P,
                                          ctypes.c_size_t, _P]),
    "la_prefix_mask": (ctypes.c_int, [ctypes.POINTER(la_desc), ctypes.c_int32, _P, _P, _P, _P, _P,
                                      _P, ctypes.c_size_t, _P]),
    "la_decode_step": (ctypes.c_int, [ctypes.POINTER(la_desc), _P, _P, _P, _P, _P, _P, _P]),
    "la_gated_causal": (ctypes.c_int, [ctypes.POINTER(la_desc)] + [_P] * 10 + [ctypes.c_size_t, _P]),
    "la_gated_causal_backward": (ctypes.c_int, [ctypes.POINTER(la_desc)] + [_P] * 10 + [ctypes.c_size_t, _P]),
    "la_gated_decode_step": (ctypes.c_int, [ctypes.POINTER(la_desc)] + [_P] * 10),
    "la_qk_norm_rope": (ctypes.c_int, _ROPE + [_P, _P, _P]),
    "la_qk_norm_rope_backward": (ctypes.c_int, _ROPE + [_P, _P, _P, ctypes.POINTER(la_strides), _P,
                                                        ctypes.POINTER(la_strides), _P, _P, _P, ctypes.c_size_t, _P]),
    "la_qk_norm_rope_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(la_rope_desc)]),
    "la_kv_summary_static": (ctypes.c_int, [ctypes.POINTER(la_desc), _P, _P, _P, _P, _P]),
    "la_last_error": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_uint32)]),
    "la_timing_enable": (ctypes.c_int, [ctypes.c_int32]),
    "la_timing_read": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float), ctypes.c_int32,
                                      ctypes.POINTER(ctypes.c_int32)]),
    "la_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "la_version": (ctypes.c_int32, []),
}


def lib():
    """The loaded library (raises if it is missing: build it first with
    ``python -m kernelized_linear_attention_phi_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libla_b200.so is not built ({LIB_PATH})")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def make_desc(B, H, N, d, dtype, phi="relu1", normalize=True) -> la_desc:
    return la_desc(int(B), int(H), int(N), int(d), DTYPES.get(dtype, dtype) if not isinstance(dtype, int) else dtype,
                   PHIS[phi] if isinstance(phi, str) else int(phi), int(bool(normalize)))


def _desc_of(x: torch.Tensor, phi, normalize) -> la_desc:
    if x.dim() != 4:
        raise ValueError(f"expected a [B, H, N, d] tensor, got shape {tuple(x.shape)}")
    if x.dtype not in DTYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    B, H, N, d = x.shape
    return make_desc(B, H, N, d, x.dtype, phi, normalize)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(t, stream):
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(fn, status):
    if status != LA_OK:
        raise LaError(fn, status)


def _same(ref, *ts):
    for t in ts:
        if t.dtype != ref.dtype or t.shape != ref.shape or t.device != ref.device:
            raise ValueError("q, k, v and out must share shape, dtype and device")


def _state(S, z, ref):
    """S [B,H,d,d] and z [B,H,d]: contiguous float32 on ref's device (the
    library writes or reads exactly that many floats)."""
    B, H, _, d = ref.shape
    if S.dtype != torch.float32 or tuple(S.shape) != (B, H, d, d) or S.device != ref.device:
        raise ValueError(f"S must be float32 [{B}, {H}, {d}, {d}] on {ref.device}")
    if z.dtype != torch.float32 or tuple(z.shape) != (B, H, d) or z.device != ref.device:
        raise ValueError(f"z must be float32 [{B}, {H}, {d}] on {ref.device}")
    if not S.is_contiguous() or not z.is_contiguous():
        raise ValueError("S and z must be contiguous")


def _ws(ws, ref):
    """A workspace: a contiguous uint8 buffer on ref's device (the library
    checks its size)."""
    if ws.dtype != torch.uint8 or ws.device != ref.device or not ws.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous uint8 tensor on {ref.device}")
    return ws


def la_version() -> int:
    return int(lib().la_version())


def la_status_string(status: int) -> str:
    return lib().la_status_string(int(status)).decode()


def la_workspace_size(desc: la_desc, op, chunk: int = 64) -> int:
    return int(lib().la_workspace_size(ctypes.byref(desc), OPS.get(op, op), int(chunk)))


def workspace(desc: la_desc, op, chunk: int = 64, device="cuda") -> torch.Tensor:
    """A device buffer big enough for ``op`` on ``desc``, with its error word
    zeroed (the library only sets bits in it; la_last_error reads and
    clears). The rest needs no initialization."""
    n = la_workspace_size(desc, op, chunk)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def la_kv_summary(k, v, S_out=None, z_out=None, phi="relu1", ws=None, stream=None):
    """S = sum_j phi(k_j) (x) v_j, z = sum_j phi(k_j) per head. Returns (S, z)."""
    _same(k, v)
    desc = _desc_of(k, phi, True)
    B, H, _, d = k.shape
    if S_out is None:
        S_out = torch.empty(B, H, d, d, dtype=torch.float32, device=k.device)
    if z_out is None:
        z_out = torch.empty(B, H, d, dtype=torch.float32, device=k.device)
    _state(S_out, z_out, k)
    ws = workspace(desc, "kv_summary", device=k.device) if ws is None else _ws(ws, k)
    _check("la_kv_summary", lib().la_kv_summary(
        ctypes.byref(desc), _ptr(k), _ptr(v), _ptr(S_out), _ptr(z_out), _ptr(ws), ws.numel(),
        _stream(k, stream)))
    return S_out, z_out


def la_kv_summary_static(k, v, S_out, z_out, phi="relu1", stream=None):
    """la_kv_summary with the library's own device scratch instead of a
    workspace: for callers that cannot allocate device memory. Allocates
    nothing; S_out [B,H,d,d] and z_out [B,H,d] float32 are the caller's.
    Calls that overlap on the GPU race (they share the scratch)."""
    _same(k, v)
    _state(S_out, z_out, k)
    desc = _desc_of(k, phi, True)
    _check("la_kv_summary_static", lib().la_kv_summary_static(
        ctypes.byref(desc), _ptr(k), _ptr(v), _ptr(S_out), _ptr(z_out), _stream(k, stream)))
    return S_out, z_out


def la_noncausal(q, k, v, out=None, S_out=None, z_out=None, phi="relu1", normalize=True, ws=None,
                 stream=None):
    """Non-causal attention. Returns out (and fills S_out/z_out if given)."""
    if out is None:
        out = torch.empty_like(q)
    _same(q, k, v, out)
    if (S_out is None) != (z_out is None):
        raise ValueError("give both S_out and z_out, or neither")
    if S_out is not None:
        _state(S_out, z_out, q)
    desc = _desc_of(q, phi, normalize)
    ws = workspace(desc, "noncausal", device=q.device) if ws is None else _ws(ws, q)
    _check("la_noncausal", lib().la_noncausal(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(S_out), _ptr(z_out),
        _ptr(ws), ws.numel(), _stream(q, stream)))
    return out


def la_causal_chunked(q, k, v, out=None, chunk=64, phi="relu1", normalize=True, ws=None,
                      stream=None):
    """Causal attention (query i sees keys 0..i). Returns out."""
    if out is None:
        out = torch.empty_like(q)
    _same(q, k, v, out)
    desc = _desc_of(q, phi, normalize)
    ws = workspace(desc, "causal", chunk, device=q.device) if ws is None else _ws(ws, q)
    _check("la_causal_chunked", lib().la_causal_chunked(
        ctypes.byref(desc), int(chunk), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(ws),
        ws.numel(), _stream(q, stream)))
    return out


def la_causal_prefill(q, k, v, out=None, S_out=None, z_out=None, chunk=64, phi="relu1", normalize=True,
                      ws=None, stream=None):
    """Causal attention plus the state after the last token (the cache a
    decode continues from). Returns (out, S, z)."""
    if out is None:
        out = torch.empty_like(q)
    _same(q, k, v, out)
    B, H, _, d = q.shape
    if S_out is None:
        S_out = torch.empty(B, H, d, d, dtype=torch.float32, device=q.device)
    if z_out is None:
        z_out = torch.empty(B, H, d, dtype=torch.float32, device=q.device)
    _state(S_out, z_out, q)
    desc = _desc_of(q, phi, normalize)
    ws = workspace(desc, "causal", chunk, device=q.device) if ws is None else _ws(ws, q)
    _check("la_causal_prefill", lib().la_causal_prefill(
        ctypes.byref(desc), int(chunk), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(S_out), _ptr(z_out),
        _ptr(ws), ws.numel(), _stream(q, stream)))
    return out, S_out, z_out


def la_prefix_mask(q, k, v, m, out=None, chunk=64, phi="relu1", normalize=True, ws=None,
                   stream=None):
    """Prefix-mask attention (query i of sequence b sees keys 0..m[b, i]). Returns out."""
    if out is None:
        out = torch.empty_like(q)
    _same(q, k, v, out)
    B, _, N, _ = q.shape
    if m.dtype != torch.int32 or tuple(m.shape) != (B, N) or m.device != q.device:
        raise ValueError("m must be an int32 [B, N] tensor on the same device")
    if not m.is_contiguous():
        raise ValueError("m must be contiguous")
    desc = _desc_of(q, phi, normalize)
    ws = workspace(desc, "prefix", chunk, device=q.device) if ws is None else _ws(ws, q)
    _check("la_prefix_mask", lib().la_prefix_mask(
        ctypes.byref(desc), int(chunk), _ptr(q), _ptr(k), _ptr(v), _ptr(m), _ptr(out), _ptr(ws),
        ws.numel(), _stream(q, stream)))
    return out


def la_decode_step(q, k, v, S, z, out=None, phi="relu1", normalize=True, stream=None):
    """One decode step on the state (S, z), updated in place. q, k, v: [B, H, 1, d]."""
    if out is None:
        out = torch.empty_like(q)
    _same(q, k, v, out)
    _state(S, z, q)
    desc = _desc_of(q, phi, normalize)
    _check("la_decode_step", lib().la_decode_step(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(S), _ptr(z), _ptr(out),
        _stream(q, stream)))
    return out


def la_last_error(ws, stream=None):
    """Synchronizes, reads and clears the workspace error word. Returns
    (status, flags)."""
    flags = ctypes.c_uint32(0)
    st = lib().la_last_error(_ptr(ws), _stream(ws, stream), ctypes.byref(flags))
    return int(st), int(flags.value)


def la_timing_enable(enable=True):
    """Turns the library's per-kernel timing events on or off (on: creates
    them on the current device)."""
    _check("la_timing_enable", lib().la_timing_enable(1 if enable else 0))


def la_timing_read(capacity=16):
    """Durations in ms of the kernels of the last timed call (or graph
    replay), in launch order; waits for that call to finish."""
    buf = (ctypes.c_float * capacity)()
    n = ctypes.c_int32(0)
    _check("la_timing_read", lib().la_timing_read(buf, capacity, ctypes.byref(n)))
    return [float(buf[i]) for i in range(min(n.value, capacity))]


def _backward(name, op, q, k, v, dout, dq, dk, dv, phi, normalize, ws, stream):
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _same(q, k, v, dout, dq, dk, dv)
    desc = _desc_of(q, phi, normalize)
    ws = workspace(desc, op, 64, device=q.device) if ws is None else _ws(ws, q)
    _check(name, getattr(lib(), name)(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
        ws.numel(), _stream(q, stream)))
    return dq, dk, dv


def la_noncausal_backward(q, k, v, dout, dq=None, dk=None, dv=None, phi="relu1", normalize=True, ws=None,
                          stream=None):
    """Gradients (dq, dk, dv) of non-causal attention for upstream dout."""
    return _backward("la_noncausal_backward", "noncausal_bwd", q, k, v, dout, dq, dk, dv, phi, normalize, ws,
                     stream)


def la_causal_backward(q, k, v, dout, dq=None, dk=None, dv=None, phi="relu1", normalize=True, ws=None,
                       stream=None):
    """Gradients (dq, dk, dv) of causal attention for upstream dout."""
    return _backward("la_causal_backward", "causal_bwd", q, k, v, dout, dq, dk, dv, phi, normalize, ws, stream)


# The entry points below take the caller's tensors as they are and check each
# once; shapes, types and devices are compared as plain tuples and numbers,
# since at one token the call is host time.


# the handle of torch's current stream, without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _on:
    """The device of a call's tensors and its stream (torch's current one there
    when None) made current: what the call allocates and clears is then ordered
    with its kernels, whatever device and stream the caller was on. Entering
    gives the stream's handle."""

    __slots__ = ("index", "guards", "stream")

    def __init__(self, ref, stream):
        self.index = ref.get_device()
        if self.index < 0:
            raise ValueError("tensors must be on a CUDA device")
        self.guards = None
        self.stream = stream

    def __enter__(self):
        if self.stream is None and self.index == torch.cuda.current_device():
            return _raw_stream(self.index)
        stream = self.stream
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=self.index)
        self.guards = [torch.cuda.device(self.index)]
        if stream is not None:
            self.guards.append(torch.cuda.stream(stream))
        for g in self.guards:
            g.__enter__()
        return _raw_stream(self.index)

    def __exit__(self, *exc):
        for g in reversed(self.guards or ()):
            g.__exit__(*exc)


def _arg(name, t, dtype, shape, index):
    """The address of a contiguous tensor of the given type, shape and device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{index}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    return t.data_ptr()


def _scratch(ref, nbytes):
    """A workspace that nobody but one call sees: its error word, which no one
    can ask for afterwards, needs no clearing. (0 bytes: a request that the
    library is about to refuse.)"""
    return ref.new_empty((max(nbytes, 16),), dtype=torch.uint8)


@functools.lru_cache(maxsize=256)
def _gated_desc(shape, dtype, phi, normalize):
    if len(shape) != 4:
        raise ValueError(f"expected a [B, H, N, d] tensor, got shape {tuple(shape)}")
    if dtype not in DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    return make_desc(*shape, dtype, phi, normalize)


def _pair(what, a, b):
    if (a is None) != (b is None):
        raise ValueError(f"give both S and z of {what}, or neither")


def la_gated_causal(q, k, v, g, S_in=None, z_in=None, out=None, S_out=None, z_out=None, phi="relu1", normalize=True,
                    ws=None, stream=None):
    """Causal attention with a decay exp(g) per head and token (g: [B, H, N]
    log-gates, -inf starts anew). S_in, z_in: the state in front of the first
    token; S_out, z_out (may be the same) receive the one after the last.
    Returns out."""
    shape, dt = q.shape, q.dtype
    desc = _gated_desc(shape, dt, phi, bool(normalize))
    _pair("the state in front", S_in, z_in)
    _pair("the state behind", S_out, z_out)
    with _on(q, stream) as st:
        i = q.get_device()
        B, H, N, d = shape
        args = [_arg("q", q, dt, shape, i), _arg("k", k, dt, shape, i), _arg("v", v, dt, shape, i),
                _arg("g", g, dt, (B, H, N), i)]
        for S, z in ((S_in, z_in), (S_out, z_out)):
            if S is None:
                args += (None, None)
            else:
                args += (_arg("S", S, torch.float32, (B, H, d, d), i), _arg("z", z, torch.float32, (B, H, d), i))
        out = torch.empty_like(q) if out is None else out
        args.insert(6, _arg("out", out, dt, shape, i))
        ws = _scratch(q, la_workspace_size(desc, "gated_causal")) if ws is None else _ws(ws, q)
        _check("la_gated_causal", lib().la_gated_causal(ctypes.byref(desc), *args, ws.data_ptr(), ws.numel(), st))
    return out


def la_gated_causal_backward(q, k, v, g, dout, dq=None, dk=None, dv=None, dg=None, phi="relu1", normalize=True, ws=None,
                             stream=None):
    """Gradients (dq, dk, dv, dg) of la_gated_causal, from an empty state, for
    upstream dout."""
    shape, dt = q.shape, q.dtype
    desc = _gated_desc(shape, dt, phi, bool(normalize))
    with _on(q, stream) as st:
        i = q.get_device()
        gates = tuple(shape[:3])
        args = [_arg("q", q, dt, shape, i), _arg("k", k, dt, shape, i), _arg("v", v, dt, shape, i),
                _arg("g", g, dt, gates, i), _arg("dout", dout, dt, shape, i)]
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        dg = torch.empty_like(g) if dg is None else dg
        args += (_arg("dq", dq, dt, shape, i), _arg("dk", dk, dt, shape, i), _arg("dv", dv, dt, shape, i),
                 _arg("dg", dg, dt, gates, i))
        ws = _scratch(q, la_workspace_size(desc, "gated_causal_bwd")) if ws is None else _ws(ws, q)
        _check("la_gated_causal_backward", lib().la_gated_causal_backward(
            ctypes.byref(desc), *args, ws.data_ptr(), ws.numel(), st))
    return dq, dk, dv, dg


def la_gated_decode_step(q, k, v, g, S, z, S_out=None, z_out=None, out=None, phi="relu1", normalize=True, stream=None):
    """One token on the state (S, z): q, k, v [B, H, 1, d], g [B, H, 1]. The new
    state goes to S_out, z_out, or in place when they are not given. Returns out."""
    shape, dt = q.shape, q.dtype
    desc = _gated_desc(shape, dt, phi, bool(normalize))
    B, H, N, d = shape
    if N != 1:
        raise ValueError("a step takes one token: [B, H, 1, d]")
    _pair("the new state", S_out, z_out)
    with _on(q, stream) as st:
        i = q.get_device()
        s = _arg("S", S, torch.float32, (B, H, d, d), i), _arg("z", z, torch.float32, (B, H, d), i)
        new = s
        if S_out is not None:
            new = _arg("S_out", S_out, torch.float32, (B, H, d, d), i), _arg("z_out", z_out, torch.float32, (B, H, d), i)
        out = torch.empty_like(q) if out is None else out
        _check("la_gated_decode_step", lib().la_gated_decode_step(
            ctypes.byref(desc), _arg("q", q, dt, shape, i), _arg("k", k, dt, shape, i), _arg("v", v, dt, shape, i),
            _arg("g", g, dt, (B, H, 1), i), *s, *new, _arg("out", out, dt, shape, i), st))
    return out


@functools.lru_cache(maxsize=256)
def _rope_desc(q_shape, k_shape, dtype, table, interleaved, eps):
    if len(q_shape) != 4 or len(k_shape) != 4 or q_shape[:2] != k_shape[:2] or q_shape[3] != k_shape[3]:
        raise ValueError(f"expected q [B, N, Hq, d] and k [B, N, Hk, d], got {tuple(q_shape)} and {tuple(k_shape)}")
    if dtype not in DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    B, N, Hq, d = q_shape
    if len(table) != 2:
        raise ValueError("cos and sin must be [rows, rot / 2] tables")
    rows, rot = table[0], 2 * table[1]
    if rows >= 1 << 31 or rot > d:
        raise ValueError(f"the tables turn {rot} of {d} channels and have {rows} rows")
    return la_rope_desc(B, N, Hq, k_shape[2], d, rot, DTYPES[dtype], int(interleaved), rows, eps)


def _rope_inputs(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved):
    """The descriptor and the arguments that both directions share."""
    if (cos is None) != (sin is None) or (q_weight is None) != (k_weight is None):
        raise ValueError("give both cos and sin, and both weights, or neither")
    table = (0, 0) if cos is None else cos.shape
    desc = _rope_desc(q.shape, k.shape, q.dtype, table, bool(interleaved), float(eps))
    i = q.get_device()
    if k.dtype is not q.dtype or k.get_device() != i:
        raise ValueError("q and k must share a device and a dtype (float32 or bfloat16)")
    B, N, _, d = q.shape
    f32 = torch.float32
    small = []
    for name, t, shape in (("q_weight", q_weight, (d,)), ("k_weight", k_weight, (d,)), ("cos", cos, table),
                           ("sin", sin, table)):
        small.append(None if t is None else _arg(name, t, f32, shape, i))
    small.append(None if positions is None else _arg("positions", positions, torch.int32, (B, N), i))
    return desc, [q.data_ptr(), _strides("q", q), k.data_ptr(), _strides("k", k), *small]


def _strides(name, t):
    """The strides of a [B, N, H, d] view with contiguous rows."""
    b, n, h, one = t.stride()
    if one != 1 and t.shape[3] != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return ctypes.byref(la_strides(b, n, h))


def la_qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions=None, eps=1e-6, interleaved=False, q_out=None,
                    k_out=None, stream=None):
    """Norm of each query and key row (float32 weights [d] or None) and the
    rotation of its first 2 * cos.shape[1] channels by its position's row of
    the tables (float32 [rows, rot / 2]; None: norm only). q [B, N, Hq, d] and
    k [B, N, Hk, d] may be views into one projection; positions int32 [B, N],
    or None for 0 .. N - 1. Returns contiguous (q_out [B, Hq, N, d], k_out
    [B, Hk, N, d])."""
    with _on(q, stream) as st:
        desc, args = _rope_inputs(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)
        i, dt = q.get_device(), q.dtype
        B, N, Hq, d = q.shape
        qs, ks = (B, Hq, N, d), (B, desc.Hk, N, d)
        q_out = q.new_empty(qs) if q_out is None else q_out
        k_out = q.new_empty(ks) if k_out is None else k_out
        _check("la_qk_norm_rope", lib().la_qk_norm_rope(
            ctypes.byref(desc), *args, _arg("q_out", q_out, dt, qs, i), _arg("k_out", k_out, dt, ks, i), st))
    return q_out, k_out


def la_qk_norm_rope_backward(q, k, q_weight, k_weight, cos, sin, dq_out, dk_out, positions=None, eps=1e-6,
                             interleaved=False, dq=None, dk=None, dq_weight=None, dk_weight=None, ws=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of la_qk_norm_rope for upstream
    dq_out [B, Hq, N, d], dk_out [B, Hk, N, d]. dq, dk may be given as views
    like q, k (of one packed gradient, say). Without weights the last two are
    None."""
    with _on(q, stream) as st:
        desc, args = _rope_inputs(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)
        i, dt = q.get_device(), q.dtype
        B, N, Hq, d = q.shape
        args += (_arg("dq_out", dq_out, dt, (B, Hq, N, d), i), _arg("dk_out", dk_out, dt, (B, desc.Hk, N, d), i))
        dq = q.new_empty(q.shape) if dq is None else dq
        dk = k.new_empty(k.shape) if dk is None else dk
        for name, t, like in (("dq", dq, q), ("dk", dk, k)):
            if t.dtype is not dt or t.shape != like.shape or t.get_device() != i:
                raise ValueError("dq and dk must have the shape, dtype and device of q and k")
            args += (t.data_ptr(), _strides(name, t))
        if q_weight is None:
            if dq_weight is not None or dk_weight is not None:
                raise ValueError("there are no weights to differentiate")
            args += (None, None)
        else:
            dq_weight = q_weight.new_empty((d,)) if dq_weight is None else dq_weight
            dk_weight = k_weight.new_empty((d,)) if dk_weight is None else dk_weight
            args += (_arg("dq_weight", dq_weight, torch.float32, (d,), i),
                     _arg("dk_weight", dk_weight, torch.float32, (d,), i))
        if ws is None:
            ws = _scratch(q, int(lib().la_qk_norm_rope_workspace_size(ctypes.byref(desc))))
        else:
            _ws(ws, q)
        _check("la_qk_norm_rope_backward", lib().la_qk_norm_rope_backward(
            ctypes.byref(desc), *args, ws.data_ptr(), ws.numel(), st))
    return dq, dk, dq_weight, dk_weight
