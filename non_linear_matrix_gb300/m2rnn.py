"""Thin ctypes binding of libm2rnn.so (include/m2rnn.h and m2rnn_block.h).

Argument marshalling only: it checks tensor placement and dtypes, allocates
output tensors with torch, passes raw device pointers and the current CUDA
stream to the C ABI and turns non-zero status codes into exceptions.  Every
step of the recurrence runs in the library's CUDA kernels; if the library is
not built this module raises instead of computing anything itself.

A call with ``stream=`` behaves as under ``torch.cuda.stream(stream)``: it is queued
there, and what it allocates is that stream's memory.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libm2rnn.so")
# The checked build (index checks in every kernel, M2RNN_ERR_BOUNDS), loaded
# instead of LIB_PATH when M2RNN_LIBRARY=checked or after use_library("checked").
LIB_CHECKED_PATH = os.path.join(_HERE, "_build", "check", "libm2rnn_check.so")

M2RNN_F32, M2RNN_BF16 = 0, 1
STATUS = {
    0: "M2RNN_OK", -1: "M2RNN_ERR_INVALID_ARG", -2: "M2RNN_ERR_UNSUPPORTED_SHAPE",
    -3: "M2RNN_ERR_MISALIGNED", -4: "M2RNN_ERR_POINTER", -5: "M2RNN_ERR_WORKSPACE",
    -6: "M2RNN_ERR_CUDA", -7: "M2RNN_ERR_TIMEOUT", -8: "M2RNN_ERR_BOUNDS",
}

_lock = threading.Lock()
_lib = None

_VP = ctypes.c_void_p
_EXPORTS = {
    "m2rnn_version": (ctypes.c_int, []),
    "m2rnn_checked": (ctypes.c_int, []),
    "m2rnn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "m2rnn_num_checkpoints": (ctypes.c_size_t, [_VP]),
    "m2rnn_fwd": (ctypes.c_int, [_VP] * 12),
    "m2rnn_bwd_workspace_size": (ctypes.c_size_t, [_VP, ctypes.c_int]),
    "m2rnn_bwd": (ctypes.c_int, [_VP] * 20 + [ctypes.c_size_t, _VP]),
    "m2rnn_device_status": (ctypes.c_int, [_VP, _VP, ctypes.c_int, _VP]),
    "m2rnn_set_wait_limit_ns": (ctypes.c_int, [ctypes.c_longlong]),
    "m2rnn_set_fault_injection": (ctypes.c_int, [ctypes.c_int]),
    "m2rnn_bwd_noalloc": (ctypes.c_int, [_VP] * 18),
    "m2rnn_decode": (ctypes.c_int, [_VP] * 11),
    "m2rnn_decode_gated": (ctypes.c_int, [_VP] * 13),
    "m2rnn_fwd_gated": (ctypes.c_int, [_VP] * 14),
    "m2rnn_bwd_gated": (ctypes.c_int, [_VP] * 24 + [ctypes.c_size_t, _VP]),
    "m2rnn_fwd_norm": (ctypes.c_int, [_VP] * 13 + [ctypes.c_float] + [_VP] * 6),
    "m2rnn_bwd_norm_workspace_size": (ctypes.c_size_t, [_VP, ctypes.c_int]),
    "m2rnn_bwd_norm": (ctypes.c_int, [_VP] * 31 + [ctypes.c_size_t, _VP]),
    "m2rnn_conv_fwd": (ctypes.c_int, [_VP] * 9),
    "m2rnn_conv_bwd_workspace_size": (ctypes.c_size_t, [_VP]),
    "m2rnn_conv_bwd": (ctypes.c_int, [_VP] * 13 + [ctypes.c_size_t, _VP]),
    "m2rnn_conv_step": (ctypes.c_int, [_VP] * 9),
    "m2rnn_qk_norm_fwd": (ctypes.c_int, [_VP] * 7 + [ctypes.c_float] + [_VP] * 6),
    "m2rnn_qk_norm_bwd_workspace_size": (ctypes.c_size_t, [_VP]),
    "m2rnn_qk_norm_bwd": (ctypes.c_int, [_VP] * 7 + [ctypes.c_float] + [_VP] * 10 +
                          [ctypes.c_size_t, _VP]),
    "m2rnn_scan_saved_size": (ctypes.c_size_t, [_VP]),
    "m2rnn_scan_fwd_workspace_size": (ctypes.c_size_t, [_VP, ctypes.c_int]),
    "m2rnn_scan_fwd": (ctypes.c_int, [_VP] * 14 + [ctypes.c_size_t, _VP]),
    "m2rnn_scan_bwd_workspace_size": (ctypes.c_size_t, [_VP, ctypes.c_int]),
    "m2rnn_scan_bwd": (ctypes.c_int, [_VP] * 22 + [ctypes.c_size_t, _VP]),
    "m2rnn_scan_step": (ctypes.c_int, [_VP] * 13),
}


class M2RNNError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)} ({status_string(code)})")


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("N", ctypes.c_int),
                ("K", ctypes.c_int), ("V", ctypes.c_int), ("in_dtype", ctypes.c_int),
                ("ckpt_every", ctypes.c_int), ("Nq", ctypes.c_int)]


def _load(path: str, how: str) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           f"`python -m non_linear_matrix_gb300.build{how}` (there is no fallback)")
    L = ctypes.CDLL(path)
    for name, (res, args) in _EXPORTS.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def lib() -> ctypes.CDLL:
    """The loaded native library (raises if it was never built)."""
    global _lib
    with _lock:
        if _lib is None:
            if os.environ.get("M2RNN_LIBRARY") == "checked":
                _lib = _load(LIB_CHECKED_PATH, " checked")
            else:
                _lib = _load(LIB_PATH, "")
    return _lib


def use_library(which: str):
    """Switch every later call to the normal ("normal") or the checked
    ("checked") build; both must have been built.  Each build keeps its own
    device status word."""
    global _lib
    if which not in ("normal", "checked"):
        raise ValueError(which)
    with _lock:
        _lib = _load(LIB_CHECKED_PATH, " checked") if which == "checked" else _load(LIB_PATH, "")


def status_string(code: int) -> str:
    return lib().m2rnn_status_string(int(code)).decode()


def _check(rc: int, where: str):
    if rc != 0:
        raise M2RNNError(rc, where)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return M2RNN_BF16
    if t.dtype == torch.float32:
        return M2RNN_F32
    raise TypeError(f"unsupported input dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libm2rnn must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libm2rnn must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _tensors(r):
    """The tensors of a call's result (a tensor, a dict or a tuple)."""
    if isinstance(r, (dict, tuple)):
        for x in r.values() if isinstance(r, dict) else r:
            yield from _tensors(x)
    elif r is not None:
        yield r


def _on_stream(call):
    """``call`` with ``stream=``: what it allocates (scratch that it drops on return,
    results) comes from that stream's own memory.  Taken from the current
    stream's, the scratch could go to the next allocation there while the call still
    works in it, or still be in use by what was queued there before.  The
    results are marked as used on the current stream too, so that the caller may drop
    them while work that was queued there reads them."""
    @functools.wraps(call)
    def on_stream(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        caller = torch.cuda.current_stream(stream.device)
        with torch.cuda.stream(stream):
            r = call(*args, stream=stream, **kw)
        if stream != caller:
            for t in _tensors(r):
                t.record_stream(caller)
        return r
    return on_stream


def make_shape(q, v, ckpt_every: int = 0) -> Shape:
    """Shape of a call; q is [B,T,K] (shared by all heads) or [B,T,Nq,K]
    (Nq query/key groups)."""
    if q.dim() == 4:
        B, T, Nq, K = q.shape
    else:
        (B, T, K), Nq = q.shape, 1
    N, V = v.shape[2], v.shape[3]
    return Shape(B, T, N, K, V, _dtype_code(q), int(ckpt_every), Nq)


def num_checkpoints(shape: Shape) -> int:
    return int(lib().m2rnn_num_checkpoints(ctypes.byref(shape)))


@_on_stream
def fwd(q, k, v, f, W, w_r, H0=None, *, ckpt_every: int = 0, want_HT: bool = True,
        out=None, stream=None):
    """Forward pass.  Returns (y, H_T or None, ckpt or None).

    q, k [B,T,K]; v [B,T,N,V]; f [B,T,N]; W [N,V,V]; w_r [N,V], all of one
    dtype (bf16 or f32); H0 [B,N,K,V] fp32 or None.  ``out`` may supply a
    dict of preallocated outputs (y, HT, ckpt)."""
    s = make_shape(q, v, ckpt_every)
    for t in (k, v, f, W, w_r):
        if t.dtype != q.dtype:
            raise TypeError("q, k, v, f, W, w_r must share one dtype")
    out = dict(out or {})
    y = out.get("y")
    if y is None:
        y = torch.empty_like(v)
    HT = out.get("HT")
    if HT is None and want_HT:
        HT = torch.empty(s.B, s.N, s.K, s.V, device=q.device, dtype=torch.float32)
    ck = out.get("ckpt")
    nck = num_checkpoints(s)
    if ck is None and nck > 0:
        ck = torch.empty(s.B, s.N, nck, s.K, s.V, device=q.device, dtype=torch.float32)
    rc = lib().m2rnn_fwd(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(f), _ptr(W), _ptr(w_r),
                         _ptr(H0), _ptr(y), _ptr(HT), _ptr(ck), _stream(stream))
    _check(rc, "m2rnn_fwd")
    return y, HT, ck


@_on_stream
def fwd_gated(q, k, v, a, alpha, beta, W, w_r, H0=None, *, ckpt_every: int = 0,
              want_HT: bool = True, out=None, stream=None):
    """Forward pass with the fused input gate f = exp(-alpha softplus(a + beta)),
    computed inside the kernel.  a [B,T,N]; alpha, beta [N]; the rest as for
    ``fwd``.  Returns (y, H_T or None, ckpt or None)."""
    s = make_shape(q, v, ckpt_every)
    for t in (k, v, a, alpha, beta, W, w_r):
        if t.dtype != q.dtype:
            raise TypeError("q, k, v, a, alpha, beta, W, w_r must share one dtype")
    out = dict(out or {})
    y = out.get("y")
    if y is None:
        y = torch.empty_like(v)
    HT = out.get("HT")
    if HT is None and want_HT:
        HT = torch.empty(s.B, s.N, s.K, s.V, device=q.device, dtype=torch.float32)
    ck = out.get("ckpt")
    nck = num_checkpoints(s)
    if ck is None and nck > 0:
        ck = torch.empty(s.B, s.N, nck, s.K, s.V, device=q.device, dtype=torch.float32)
    rc = lib().m2rnn_fwd_gated(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(alpha),
                               _ptr(beta), _ptr(W), _ptr(w_r), _ptr(H0), _ptr(y), _ptr(HT),
                               _ptr(ck), _stream(stream))
    _check(rc, "m2rnn_fwd_gated")
    return y, HT, ck


@_on_stream
def decode(q, k, v, f, W, w_r, H, *, H_out=None, y=None, stream=None):
    """One decode step for B sequences.  Returns (y, H_out).

    q, k [B,K] (or [B,Nq,K] with Nq query/key groups); v [B,N,V]; f [B,N];
    W [N,V,V]; w_r [N,V], one dtype (bf16 or f32); H [B,N,K,V] fp32 is the
    state before the step.  H_out defaults to a new tensor; pass ``H_out=H``
    to update the state in place."""
    if q.dim() == 3:
        B, Nq, K = q.shape
    else:
        (B, K), Nq = q.shape, 1
    N, V = v.shape[1], v.shape[2]
    for t in (k, v, f, W, w_r):
        if t.dtype != q.dtype:
            raise TypeError("q, k, v, f, W, w_r must share one dtype")
    s = Shape(B, 1, N, K, V, _dtype_code(q), 0, Nq)
    if H_out is None:
        H_out = torch.empty_like(H)
    if y is None:
        y = torch.empty_like(v)
    rc = lib().m2rnn_decode(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(f), _ptr(W),
                            _ptr(w_r), _ptr(H), _ptr(H_out), _ptr(y), _stream(stream))
    _check(rc, "m2rnn_decode")
    return y, H_out


@_on_stream
def decode_gated(q, k, v, a, alpha, beta, W, w_r, H, *, H_out=None, y=None, stream=None):
    """One decode step with the fused input gate: a [B,N], alpha and beta
    [N] replace f; otherwise as ``decode``.  Returns (y, H_out)."""
    if q.dim() == 3:
        B, Nq, K = q.shape
    else:
        (B, K), Nq = q.shape, 1
    N, V = v.shape[1], v.shape[2]
    for t in (k, v, a, alpha, beta, W, w_r):
        if t.dtype != q.dtype:
            raise TypeError("q, k, v, a, alpha, beta, W, w_r must share one dtype")
    s = Shape(B, 1, N, K, V, _dtype_code(q), 0, Nq)
    if H_out is None:
        H_out = torch.empty_like(H)
    if y is None:
        y = torch.empty_like(v)
    rc = lib().m2rnn_decode_gated(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(alpha),
                                  _ptr(beta), _ptr(W), _ptr(w_r), _ptr(H), _ptr(H_out), _ptr(y),
                                  _stream(stream))
    _check(rc, "m2rnn_decode_gated")
    return y, H_out


def bwd_workspace_size(shape: Shape, ckpt_given: bool) -> int:
    return int(lib().m2rnn_bwd_workspace_size(ctypes.byref(shape), int(bool(ckpt_given))))


@_on_stream
def bwd(q, k, v, f, W, w_r, dy, H0=None, ckpt=None, dHT=None, *, ckpt_every: int = 64,
        want_dH0: bool = False, want_dckpt: bool = False, workspace=None, out=None,
        stream=None):
    """BPTT backward.  Returns dict(dq, dk, dv, df, dW, dw_r[, dH0][, dckpt]) (fp32).

    ``dckpt`` is dL/dH at every checkpoint ([B,N,nck,K,V])."""
    s = make_shape(q, v, ckpt_every)
    dev = q.device
    f32 = dict(device=dev, dtype=torch.float32)
    out = dict(out or {})
    g = {
        "dq": out.get("dq"), "dk": out.get("dk"), "dv": out.get("dv"), "df": out.get("df"),
        "dW": out.get("dW"), "dw_r": out.get("dw_r"),
    }
    shapes = {"dq": tuple(q.shape), "dk": tuple(q.shape), "dv": (s.B, s.T, s.N, s.V),
              "df": (s.B, s.T, s.N), "dW": (s.N, s.V, s.V), "dw_r": (s.N, s.V)}
    for name, shp in shapes.items():
        if g[name] is None:
            g[name] = torch.empty(shp, **f32)
    dH0 = out.get("dH0")
    if dH0 is None and want_dH0:
        dH0 = torch.empty(s.B, s.N, s.K, s.V, **f32)
    dck = out.get("dckpt")
    if dck is None and want_dckpt:
        dck = torch.empty(s.B, s.N, num_checkpoints(s), s.K, s.V, **f32)
    need = bwd_workspace_size(s, ckpt is not None)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=dev, dtype=torch.uint8)
    rc = lib().m2rnn_bwd(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(f), _ptr(W), _ptr(w_r),
                         _ptr(H0), _ptr(ckpt), _ptr(dy), _ptr(dHT),
                         _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["df"]),
                         _ptr(g["dW"]), _ptr(g["dw_r"]), _ptr(dH0), _ptr(dck), _ptr(workspace),
                         ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check(rc, "m2rnn_bwd")
    if dH0 is not None:
        g["dH0"] = dH0
    if dck is not None:
        g["dckpt"] = dck
    return g


@_on_stream
def bwd_noalloc(q, k, v, f, W, w_r, dy, H0=None, dHT=None, *, ckpt_every: int = 64,
                want_dH0: bool = False, out=None, stream=None):
    """Backward pass that allocates nothing inside the library (checkpoints
    are recomputed into a buffer built into it).  Same outputs as
    ``bwd(..., ckpt=None)``; output tensors come from ``out`` or are created
    here by the caller side."""
    s = make_shape(q, v, ckpt_every)
    f32 = dict(device=q.device, dtype=torch.float32)
    out = dict(out or {})
    shapes = {"dq": tuple(q.shape), "dk": tuple(q.shape), "dv": (s.B, s.T, s.N, s.V),
              "df": (s.B, s.T, s.N), "dW": (s.N, s.V, s.V), "dw_r": (s.N, s.V)}
    g = {n: out.get(n) if out.get(n) is not None else torch.empty(shp, **f32)
         for n, shp in shapes.items()}
    dH0 = out.get("dH0")
    if dH0 is None and want_dH0:
        dH0 = torch.empty(s.B, s.N, s.K, s.V, **f32)
    rc = lib().m2rnn_bwd_noalloc(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(f), _ptr(W),
                                 _ptr(w_r), _ptr(H0), _ptr(dy), _ptr(dHT), _ptr(g["dq"]),
                                 _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["df"]), _ptr(g["dW"]),
                                 _ptr(g["dw_r"]), _ptr(dH0), _stream(stream))
    _check(rc, "m2rnn_bwd_noalloc")
    if dH0 is not None:
        g["dH0"] = dH0
    return g


@_on_stream
def bwd_gated(q, k, v, a, alpha, beta, W, w_r, dy, H0=None, ckpt=None, dHT=None, *,
              ckpt_every: int = 64, want_dH0: bool = False, want_dckpt: bool = False,
              workspace=None, out=None, stream=None):
    """BPTT backward through the fused input gate.  Returns dict(dq, dk, dv,
    da, dalpha, dbeta, dW, dw_r[, dH0][, dckpt]) (fp32); ``ckpt`` must come
    from ``fwd_gated`` with the same inputs."""
    s = make_shape(q, v, ckpt_every)
    f32 = dict(device=q.device, dtype=torch.float32)
    out = dict(out or {})
    shapes = {"dq": tuple(q.shape), "dk": tuple(q.shape), "dv": (s.B, s.T, s.N, s.V),
              "da": (s.B, s.T, s.N), "dalpha": (s.N,), "dbeta": (s.N,),
              "dW": (s.N, s.V, s.V), "dw_r": (s.N, s.V)}
    g = {n: out.get(n) if out.get(n) is not None else torch.empty(shp, **f32)
         for n, shp in shapes.items()}
    dH0 = out.get("dH0")
    if dH0 is None and want_dH0:
        dH0 = torch.empty(s.B, s.N, s.K, s.V, **f32)
    dck = out.get("dckpt")
    if dck is None and want_dckpt:
        dck = torch.empty(s.B, s.N, num_checkpoints(s), s.K, s.V, **f32)
    need = bwd_workspace_size(s, ckpt is not None)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    rc = lib().m2rnn_bwd_gated(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(alpha),
                               _ptr(beta), _ptr(W), _ptr(w_r), _ptr(H0), _ptr(ckpt), _ptr(dy),
                               _ptr(dHT), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]),
                               _ptr(g["da"]), _ptr(g["dalpha"]), _ptr(g["dbeta"]), _ptr(g["dW"]),
                               _ptr(g["dw_r"]), _ptr(dH0), _ptr(dck), _ptr(workspace),
                               ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check(rc, "m2rnn_bwd_gated")
    if dH0 is not None:
        g["dH0"] = dH0
    if dck is not None:
        g["dckpt"] = dck
    return g


@_on_stream
def fwd_norm(q, k, v, f, W, w_r, g, w_norm, eps: float = 0.0, H0=None, *, gate=None,
             ckpt_every: int = 0, want_HT: bool = True, out=None, stream=None):
    """Forward pass with the readout epilogue out = w_norm (.) (y (.) g) rstd,
    rstd = (mean over the token's N*V features of (y (.) g)^2 + eps)^(-1/2).
    ``gate=(a, alpha, beta)`` replaces f (pass f=None).  Returns dict(y, out,
    rstd, HT, ckpt)."""
    s = make_shape(q, v, ckpt_every)
    a, alpha, beta = gate if gate is not None else (None, None, None)
    out = dict(out or {})
    r = {"y": out.get("y"), "out": out.get("out"), "rstd": out.get("rstd"),
         "HT": out.get("HT"), "ckpt": out.get("ckpt")}
    if r["y"] is None:
        r["y"] = torch.empty_like(v)
    if r["out"] is None:
        r["out"] = torch.empty_like(v)
    if r["rstd"] is None:
        r["rstd"] = torch.empty(s.B, s.T, device=q.device, dtype=torch.float32)
    if r["HT"] is None and want_HT:
        r["HT"] = torch.empty(s.B, s.N, s.K, s.V, device=q.device, dtype=torch.float32)
    nck = num_checkpoints(s)
    if r["ckpt"] is None and nck > 0:
        r["ckpt"] = torch.empty(s.B, s.N, nck, s.K, s.V, device=q.device, dtype=torch.float32)
    rc = lib().m2rnn_fwd_norm(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(f), _ptr(a),
                              _ptr(alpha), _ptr(beta), _ptr(W), _ptr(w_r), _ptr(H0), _ptr(g),
                              _ptr(w_norm), ctypes.c_float(eps), _ptr(r["y"]), _ptr(r["out"]),
                              _ptr(r["rstd"]), _ptr(r["HT"]), _ptr(r["ckpt"]), _stream(stream))
    _check(rc, "m2rnn_fwd_norm")
    return r


@_on_stream
def bwd_norm(q, k, v, f, W, w_r, g, w_norm, y, rstd, dout, H0=None, ckpt=None, dHT=None, *,
             gate=None, ckpt_every: int = 64, want_dH0: bool = False, want_dckpt: bool = False,
             workspace=None, out=None, stream=None):
    """Backward pass through the readout epilogue and the recurrence.
    Returns dict(dq, dk, dv, df | da+dalpha+dbeta, dW, dw_r, dg, dw_norm
    [, dH0][, dckpt]) (fp32)."""
    s = make_shape(q, v, ckpt_every)
    a, alpha, beta = gate if gate is not None else (None, None, None)
    f32 = dict(device=q.device, dtype=torch.float32)
    out = dict(out or {})
    shapes = {"dq": tuple(q.shape), "dk": tuple(q.shape), "dv": (s.B, s.T, s.N, s.V),
              "dW": (s.N, s.V, s.V), "dw_r": (s.N, s.V), "dg": (s.B, s.T, s.N, s.V),
              "dw_norm": (s.N, s.V)}
    if gate is None:
        shapes["df"] = (s.B, s.T, s.N)
    else:
        shapes.update(da=(s.B, s.T, s.N), dalpha=(s.N,), dbeta=(s.N,))
    gr = {n: out.get(n) if out.get(n) is not None else torch.empty(shp, **f32)
          for n, shp in shapes.items()}
    dH0 = out.get("dH0")
    if dH0 is None and want_dH0:
        dH0 = torch.empty(s.B, s.N, s.K, s.V, **f32)
    dck = out.get("dckpt")
    if dck is None and want_dckpt:
        dck = torch.empty(s.B, s.N, num_checkpoints(s), s.K, s.V, **f32)
    need = int(lib().m2rnn_bwd_norm_workspace_size(ctypes.byref(s), int(ckpt is not None)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    dfa = gr["df"] if gate is None else gr["da"]
    rc = lib().m2rnn_bwd_norm(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(f), _ptr(a),
                              _ptr(alpha), _ptr(beta), _ptr(W), _ptr(w_r), _ptr(H0), _ptr(ckpt),
                              _ptr(g), _ptr(w_norm), _ptr(y), _ptr(rstd), _ptr(dout), _ptr(dHT),
                              _ptr(gr["dq"]), _ptr(gr["dk"]), _ptr(gr["dv"]), _ptr(dfa),
                              _ptr(gr.get("dalpha")), _ptr(gr.get("dbeta")), _ptr(gr["dW"]),
                              _ptr(gr["dw_r"]), _ptr(gr["dg"]), _ptr(gr["dw_norm"]), _ptr(dH0),
                              _ptr(dck), _ptr(workspace), ctypes.c_size_t(workspace.numel()),
                              _stream(stream))
    _check(rc, "m2rnn_bwd_norm")
    if dH0 is not None:
        gr["dH0"] = dH0
    if dck is not None:
        gr["dckpt"] = dck
    return gr


# ---- the operators around the recurrence (include/m2rnn_block.h) -----------


class Rows(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_longlong), ("token", ctypes.c_longlong)]


class ConvShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("C", ctypes.c_int), ("W", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int), ("silu", ctypes.c_int)]


class QkShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Nq", ctypes.c_int),
                ("Nk", ctypes.c_int), ("K", ctypes.c_int), ("R", ctypes.c_int),
                ("P", ctypes.c_int), ("in_dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int),
                ("interleaved", ctypes.c_int)]


class ScanRows(ctypes.Structure):
    _fields_ = [("q", Rows), ("k", Rows), ("v", Rows), ("a", Rows)]


def _rows(t, lead: int) -> Rows:
    """Batch and token distances of a tensor whose first ``lead`` dimensions
    are batch (and token) and whose remaining ones are packed."""
    if not t.is_cuda:
        raise ValueError("tensors passed to libm2rnn must be CUDA tensors")
    shape, st, inner = t.shape, t.stride(), 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if st[i] != inner and shape[i] != 1:
            raise ValueError("the dimensions after the token must be packed")
        inner *= shape[i]
    if lead == 1:
        return Rows(st[0] if shape[0] > 1 else inner, inner)
    token = st[1] if shape[1] > 1 else inner
    return Rows(st[0] if shape[0] > 1 else token * shape[1], token)


def _row_arg(t, lead: int):
    """The ``m2rnn_rows`` argument of an input: None where it is contiguous."""
    if t.is_contiguous() and t.is_cuda:
        return None
    return ctypes.byref(_rows(t, lead))


def _at(t):
    """Address of a tensor whose layout ``_row_arg`` or ``_rows`` checked."""
    return None if t is None else t.data_ptr()


def _addr(t):
    """Address of a tensor that must be contiguous; that it is device memory
    the library checks (M2RNN_ERR_POINTER)."""
    if t is None:
        return None
    if t.is_contiguous():
        return t.data_ptr()
    raise ValueError("tensors passed to libm2rnn must be contiguous")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(stream, t):
    """Handle of ``stream``, or of the current stream of t's device."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:  # a tenth of the time that building a Stream object takes
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _expect(name: str, t, shape, *dtypes):
    if t is None:
        return
    if t.shape != shape:  # (a torch.Size equals a tuple)
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")


def _expect_all(dtype, *specs):
    """``_expect`` for (name, tensor, shape) triples of one dtype; cheap when
    they are right."""
    for name, t, shape in specs:
        if t is not None and (t.dtype is not dtype or t.shape != shape):
            _expect(name, t, shape, dtype)


def _given(out, *names):
    """The named outputs that the caller supplied (None where not)."""
    return [None] * len(names) if out is None else [out.get(n) for n in names]


def _out(t, shape, dtype, device, name: str = "out"):
    if t is None:
        return torch.empty(shape, device=device, dtype=dtype)
    _expect(name, t, shape, dtype)
    return t


def _workspace(ws, need: int, device):
    return torch.empty(max(need, 16), device=device, dtype=torch.uint8) if ws is None else ws


def _nbytes(t):
    return ctypes.c_size_t(t.numel() * t.element_size())


def _grad_code(dy, x) -> int:
    if dy.dtype not in (torch.float32, x.dtype):
        raise TypeError("the incoming gradient must be float32 or of the inputs' dtype")
    return _dtype_code(dy)


@_on_stream
def conv_fwd(x, w, bias=None, state=None, *, silu: bool = True, want_state: bool = True,
             out=None, stream=None):
    """Short causal convolution along time with SiLU (or none, silu=False).
    Returns (y, state_out or None).

    x [B,T,C] (its rows may be a slice of a wider buffer); w [C,W], W = 2..4;
    bias [C] or None; state [B,W-1,C], the inputs before the call, or None
    for zeros; one dtype (bf16 or f32).  ``out`` may supply y and state."""
    (B, T, C), W = x.shape, w.shape[1]
    _expect_all(x.dtype, ("w", w, (C, W)), ("bias", bias, (C,)), ("state", state, (B, W - 1, C)))
    y, so = _given(out, "y", "state")
    y = _out(y, (B, T, C), x.dtype, x.device, "y")
    if so is not None or want_state:
        so = _out(so, (B, W - 1, C), x.dtype, x.device, "state")
    s = ConvShape(B, T, C, W, _dtype_code(x), 0, int(bool(silu)))
    rc = lib().m2rnn_conv_fwd(ctypes.byref(s), _at(x), _row_arg(x, 2), _addr(w), _addr(bias),
                              _addr(state), _addr(y), _addr(so), _stream_of(stream, x))
    _check(rc, "m2rnn_conv_fwd")
    return y, so


@_on_stream
def conv_bwd(x, w, dy, bias=None, state=None, dstate_out=None, *, silu: bool = True,
             want_dstate: bool = False, workspace=None, out=None, stream=None):
    """Gradient of ``conv_fwd``: dict(dx, dw, dbias[, dstate]).  dy [B,T,C]
    is float32 or of x's dtype; dstate_out [B,W-1,C] is the gradient of the
    returned state (None = 0).  dx and dstate have x's dtype, dw and dbias
    are fp32 (dbias None without a bias)."""
    (B, T, C), W = x.shape, w.shape[1]
    _expect_all(x.dtype, ("w", w, (C, W)), ("bias", bias, (C,)), ("state", state, (B, W - 1, C)),
                ("dstate_out", dstate_out, (B, W - 1, C)))
    _expect("dy", dy, (B, T, C), torch.float32, x.dtype)
    s = ConvShape(B, T, C, W, _dtype_code(x), _grad_code(dy, x), int(bool(silu)))
    dev, f32 = x.device, torch.float32
    dx, dw, db, ds = _given(out, "dx", "dw", "dbias", "dstate")
    g = {"dx": _out(dx, (B, T, C), x.dtype, dev, "dx"), "dw": _out(dw, (C, W), f32, dev, "dw"),
         "dbias": None if bias is None else _out(db, (C,), f32, dev, "dbias")}
    if ds is not None or want_dstate:
        ds = _out(ds, (B, W - 1, C), x.dtype, dev, "dstate")
    ws = _workspace(workspace, int(lib().m2rnn_conv_bwd_workspace_size(ctypes.byref(s))), dev)
    rc = lib().m2rnn_conv_bwd(ctypes.byref(s), _at(x), _row_arg(x, 2), _addr(w), _addr(bias),
                              _addr(state), _addr(dy), _addr(dstate_out), _addr(g["dx"]),
                              _addr(g["dw"]), _addr(g["dbias"]), _addr(ds), _addr(ws), _nbytes(ws),
                              _stream_of(stream, x))
    _check(rc, "m2rnn_conv_bwd")
    if ds is not None:
        g["dstate"] = ds
    return g


@_on_stream
def conv_step(x, w, state, bias=None, *, silu: bool = True, state_out=None, y=None, stream=None):
    """One token of the convolution for B sequences: x [B,C], state
    [B,W-1,C].  Returns (y, state_out); pass ``state_out=state`` to update
    the state in place."""
    (B, C), W = x.shape, w.shape[1]
    _expect_all(x.dtype, ("w", w, (C, W)), ("bias", bias, (C,)), ("state", state, (B, W - 1, C)))
    y = _out(y, (B, C), x.dtype, x.device, "y")
    so = _out(state_out, (B, W - 1, C), x.dtype, x.device, "state_out")
    s = ConvShape(B, 1, C, W, _dtype_code(x), 0, int(bool(silu)))
    rc = lib().m2rnn_conv_step(ctypes.byref(s), _at(x), _row_arg(x, 1), _addr(w), _addr(bias),
                               _addr(state), _addr(y), _addr(so), _stream_of(stream, x))
    _check(rc, "m2rnn_conv_step")
    return y, so


def _bad_qk():
    raise ValueError("q must be [B,T,Nq,K] and k [B,T,Nk,K]")


def _qk_args(q, k, wq, wk, cos, sin, pos, interleaved, grad_code):
    """Shape, rows and checked arguments shared by both directions."""
    B, T, Nq, K = q.shape if q.dim() == 4 else _bad_qk()
    Nk = 0
    if k is not None:
        if k.dim() != 4 or k.shape[:2] != q.shape[:2] or k.shape[3] != K:
            _bad_qk()
        if k.dtype is not q.dtype:
            raise TypeError("q and k must share one dtype")
        Nk = k.shape[2]
    R = P = 0
    if cos is not None or sin is not None:
        if cos is None or sin is None:
            raise ValueError("cos and sin come together")
        P, half = cos.shape
        R = 2 * half
        _expect_all(torch.float32, ("cos", cos, (P, half)), ("sin", sin, (P, half)))
    if pos is not None:
        _expect("pos", pos, (B, T), torch.int32)
    _expect_all(q.dtype, ("wq", wq, (K,)), ("wk", wk, (K,)))
    s = QkShape(B, T, Nq, Nk, K, R, P, _dtype_code(q), grad_code, int(bool(interleaved)))
    return s, _row_arg(q, 2), None if k is None else _row_arg(k, 2)


@_on_stream
def qk_norm_fwd(q, k, wq=None, wk=None, eps: float = 1e-6, *, cos=None, sin=None, pos=None,
                interleaved: bool = False, out=None, stream=None):
    """RMS norm of every query and key head over its K features, times wq /
    wk [K] (None = 1), with the first R = 2*cos.shape[1] features rotated by
    the token's angles in the same pass.  Returns (q', k').

    q [B,T,Nq,K], k [B,T,Nk,K] or None (rows may be slices); cos, sin [P,R/2]
    fp32; pos [B,T] int32 (None: token t has position t); interleaved: pairs
    (2i, 2i+1) instead of (i, i + R/2).  A position outside the table gives
    NaN and sets M2RNN_ERR_BOUNDS in the device status."""
    s, rq, rk = _qk_args(q, k, wq, wk, cos, sin, pos, interleaved, 0)
    qo, ko = _given(out, "q", "k")
    qo = _out(qo, q.shape, q.dtype, q.device, "q")
    ko = None if k is None else _out(ko, k.shape, q.dtype, q.device, "k")
    rc = lib().m2rnn_qk_norm_fwd(ctypes.byref(s), _at(q), rq, _at(k), rk,
                                  _addr(wq), _addr(wk), eps,
                                 _addr(cos), _addr(sin), _addr(pos), _addr(qo), _addr(ko),
                                 _stream_of(stream, q))
    _check(rc, "m2rnn_qk_norm_fwd")
    return qo, ko


@_on_stream
def qk_norm_bwd(q, k, wq, wk, dqo, dko, eps: float = 1e-6, *, cos=None, sin=None, pos=None,
                interleaved: bool = False, workspace=None, out=None, stream=None):
    """Gradient of ``qk_norm_fwd``: dict(dq, dk, dwq, dwk); dqo, dko are
    float32 or of q's dtype, dq and dk have q's dtype, dwq and dwk [K] are
    fp32 (None without that weight)."""
    s, rq, rk = _qk_args(q, k, wq, wk, cos, sin, pos, interleaved, _grad_code(dqo, q))
    _expect("dqo", dqo, q.shape, torch.float32, q.dtype)
    if (k is None) != (dko is None):
        raise ValueError("dko goes with k")
    if k is not None:
        _expect("dko", dko, k.shape, dqo.dtype)
    dev, K = q.device, q.shape[3]
    dq, dk, dwq, dwk = _given(out, "dq", "dk", "dwq", "dwk")
    g = {"dq": _out(dq, q.shape, q.dtype, dev, "dq"),
         "dk": None if k is None else _out(dk, k.shape, q.dtype, dev, "dk"),
         "dwq": None if wq is None else _out(dwq, (K,), torch.float32, dev, "dwq"),
         "dwk": None if wk is None else _out(dwk, (K,), torch.float32, dev, "dwk")}
    ws = _workspace(workspace, int(lib().m2rnn_qk_norm_bwd_workspace_size(ctypes.byref(s))), dev)
    rc = lib().m2rnn_qk_norm_bwd(ctypes.byref(s), _at(q), rq, _at(k), rk,
                                  _addr(wq), _addr(wk), eps,
                                 _addr(cos), _addr(sin), _addr(pos), _addr(dqo), _addr(dko),
                                 _addr(g["dq"]), _addr(g["dk"]), _addr(g["dwq"]), _addr(g["dwk"]),
                                 _addr(ws), _nbytes(ws), _stream_of(stream, q))
    _check(rc, "m2rnn_qk_norm_bwd")
    return g


def _scan_args(q, k, v, a, alpha, beta, w_r, lead: int):
    """Shape and rows of a scan call; q, k may lack the group dimension."""
    first = tuple(q.shape[:lead])
    B, T = first if lead == 2 else (first[0], 1)
    Nq, K = q.shape[lead:] if q.dim() == lead + 2 else (1, *q.shape[lead:])
    N, V = v.shape[lead:]
    _expect_all(q.dtype, ("k", k, q.shape), ("v", v, (*first, N, V)), ("a", a, (*first, N)),
                ("alpha", alpha, (N,)), ("beta", beta, (N,)), ("w_r", w_r, (N, V)))
    rows = None
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and a.is_contiguous()
            and q.is_cuda):
        rows = ctypes.byref(ScanRows(_rows(q, lead), _rows(k, lead), _rows(v, lead),
                                     _rows(a, lead)))
    return Shape(B, T, N, K, V, _dtype_code(q), 0, Nq), rows


@_on_stream
def scan_fwd(q, k, v, a, alpha, beta, w_r=None, H0=None, *, want_HT: bool = True,
             save: bool = False, workspace=None, out=None, stream=None):
    """Selective scan H_t = exp(-alpha dt_t) H_{t-1} + dt_t k_t v_t^T, dt =
    softplus(a + beta), y_t = H_t^T q_t + w_r (.) v_t.  Returns (y, H_T or
    None, saved or None).

    q, k [B,T,K] or [B,T,Nq,K]; v [B,T,N,V]; a [B,T,N] (rows may be slices
    of a wider buffer); alpha, beta [N]; w_r [N,V] or None; H0 [B,N,K,V] fp32
    or None.  save=True keeps what ``scan_bwd`` would otherwise recompute (an
    opaque buffer).  ``out`` may supply y, HT and saved.  ``workspace``: at
    least m2rnn_scan_fwd_workspace_size bytes (none when saved is kept); with
    m2rnn_scan_saved_size bytes the call runs in one part."""
    s, rows = _scan_args(q, k, v, a, alpha, beta, w_r, 2)
    state, dev = (s.B, s.N, s.K, s.V), q.device
    _expect("H0", H0, state, torch.float32)
    y, HT, saved = _given(out, "y", "HT", "saved")
    y = _out(y, v.shape, q.dtype, dev, "y")
    if HT is not None or want_HT:
        HT = _out(HT, state, torch.float32, dev, "HT")
    L = lib()
    if saved is None and save:
        saved = torch.empty(max(int(L.m2rnn_scan_saved_size(ctypes.byref(s))), 16), device=dev,
                            dtype=torch.uint8)
    elif saved is not None and saved.numel() < int(L.m2rnn_scan_saved_size(ctypes.byref(s))):
        raise ValueError("saved is smaller than m2rnn_scan_saved_size")
    # (as much as runs in one part; m2rnn_scan_fwd_workspace_size is the least)
    need = int(L.m2rnn_scan_saved_size(ctypes.byref(s))) if saved is None and workspace is None else 0
    ws = _workspace(workspace, need, dev)
    rc = L.m2rnn_scan_fwd(ctypes.byref(s), rows, _at(q), _at(k), _at(v), _at(a),
                          _addr(alpha), _addr(beta), _addr(w_r), _addr(H0), _addr(y), _addr(HT),
                          _addr(saved), _addr(ws), _nbytes(ws), _stream_of(stream, q))
    _check(rc, "m2rnn_scan_fwd")
    return y, HT, saved


@_on_stream
def scan_bwd(q, k, v, a, alpha, beta, dy, w_r=None, H0=None, dHT=None, *, saved=None,
             want_dH0: bool = False, workspace=None, out=None, stream=None):
    """Gradient of ``scan_fwd`` for dL/dy = dy (v's dtype) and dL/dH_T = dHT
    (fp32 or None): dict(dq, dk, dv, da (the inputs' dtype), dalpha, dbeta,
    dw_r (fp32; None without w_r)[, dH0]).  ``saved`` comes from
    ``scan_fwd(..., save=True)`` on the same inputs; without it the forward
    states are computed again."""
    s, rows = _scan_args(q, k, v, a, alpha, beta, w_r, 2)
    state, dev, f32 = (s.B, s.N, s.K, s.V), q.device, torch.float32
    _expect_all(f32, ("H0", H0, state), ("dHT", dHT, state))
    _expect("dy", dy, v.shape, q.dtype)
    L = lib()
    dq, dk, dv, da, dal, dbe, dw, dH0 = _given(out, "dq", "dk", "dv", "da", "dalpha", "dbeta",
                                               "dw_r", "dH0")
    g = {"dq": _out(dq, q.shape, q.dtype, dev, "dq"), "dk": _out(dk, q.shape, q.dtype, dev, "dk"),
         "dv": _out(dv, v.shape, q.dtype, dev, "dv"), "da": _out(da, a.shape, q.dtype, dev, "da"),
         "dalpha": _out(dal, alpha.shape, f32, dev, "dalpha"),
         "dbeta": _out(dbe, beta.shape, f32, dev, "dbeta"),
         "dw_r": None if w_r is None else _out(dw, w_r.shape, f32, dev, "dw_r")}
    if dH0 is not None or want_dH0:
        dH0 = _out(dH0, state, f32, dev, "dH0")
    if saved is not None and saved.numel() < int(L.m2rnn_scan_saved_size(ctypes.byref(s))):
        raise ValueError("saved is smaller than m2rnn_scan_saved_size")
    ws = _workspace(workspace, int(L.m2rnn_scan_bwd_workspace_size(ctypes.byref(s),
                                                                   int(saved is not None))), dev)
    rc = L.m2rnn_scan_bwd(ctypes.byref(s), rows, _at(q), _at(k), _at(v), _at(a),
                          _addr(alpha), _addr(beta), _addr(w_r), _addr(H0), _addr(saved), _addr(dy),
                          _addr(dHT), _addr(g["dq"]), _addr(g["dk"]), _addr(g["dv"]), _addr(g["da"]),
                          _addr(g["dalpha"]), _addr(g["dbeta"]), _addr(g["dw_r"]), _addr(dH0),
                          _addr(ws), _nbytes(ws), _stream_of(stream, q))
    _check(rc, "m2rnn_scan_bwd")
    if dH0 is not None:
        g["dH0"] = dH0
    return g


@_on_stream
def scan_step(q, k, v, a, alpha, beta, H, w_r=None, *, H_out=None, y=None, stream=None):
    """One token of the selective scan for B sequences.  Returns (y, H_out).

    q, k [B,K] or [B,Nq,K]; v [B,N,V]; a [B,N] (rows may be slices); alpha,
    beta [N]; w_r [N,V] or None; H [B,N,K,V] fp32 is the state before the
    token.  Pass ``H_out=H`` to update it in place."""
    s, rows = _scan_args(q, k, v, a, alpha, beta, w_r, 1)
    state = (s.B, s.N, s.K, s.V)
    _expect("H", H, state, torch.float32)
    H_out = _out(H_out, state, torch.float32, q.device, "H_out")
    y = _out(y, v.shape, q.dtype, q.device, "y")
    rc = lib().m2rnn_scan_step(ctypes.byref(s), rows, _at(q), _at(k), _at(v),
                               _at(a), _addr(alpha), _addr(beta), _addr(w_r), _addr(H), _addr(H_out),
                               _addr(y), _stream_of(stream, q))
    _check(rc, "m2rnn_scan_step")
    return y, H_out


def device_status(clear: bool = True, stream=None):
    """(status, detail) of the device status word; synchronises the stream."""
    st, de = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().m2rnn_device_status(ctypes.byref(st), ctypes.byref(de), int(clear),
                                     _stream(stream)), "m2rnn_device_status")
    return st.value, de.value


def set_wait_limit_ns(limit_ns: int):
    _check(lib().m2rnn_set_wait_limit_ns(int(limit_ns)), "m2rnn_set_wait_limit_ns")


def set_fault_injection(mode: int):
    """Test hook: 1 makes kernels start no input transfers (time-out path)."""
    _check(lib().m2rnn_set_fault_injection(int(mode)), "m2rnn_set_fault_injection")
