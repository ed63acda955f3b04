"""Thin Python binding of libmsa.so (C ABI in include/msa.h).

Argument marshalling only: every step of the method runs in the CUDA library.  PyTorch supplies
device memory (tensors and the workspace) and the current stream.  There is no fallback: if the
library is missing or fails to load, every call raises.

Entry points (same names as the C ABI):
  msa_forward, msa_backward, msa_warmup_forward, msa_warmup_backward, msa_device_status,
  msa_workspace_size.
And the autograd pair mirroring the package API of Flash-MSA (``flash_msa_func`` /
``flash_msa_warmup_func``, PyPI page "Usage"): ``msa_func`` and ``msa_warmup_func`` return
``(attn_out, kl_loss)`` where kl_loss is a zero placeholder whose gradient drives the proxy
heads in the backward.

What stands around sparse attention in a model:
  msa_norm_rope_forward, msa_norm_rope_backward, msa_norm_rope_append (norm and rotation of the
  heads, the last one into the decode caches), with the autograd functions msa_norm_rope_func and
  msa_norm_rope_packed_func;
  msa_window_forward, msa_window_backward, msa_window_decode (causal attention over a sliding window
  and the first tokens), with the autograd function msa_window_func;
  msa_packed_plan, msa_packed_forward, msa_packed_backward (causal attention over packed sequences of
  different lengths), with the autograd function msa_packed_func;
  msa_q4_cache, msa_q4_read, msa_window_decode_q4, msa_decode_q4 (K and V caches in 4 bits, which
  msa_norm_rope_append writes too).
"""
from __future__ import annotations

import array
import ctypes
import functools
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmsa.so")

OP_FORWARD, OP_BACKWARD, OP_WARMUP_FORWARD, OP_WARMUP_BACKWARD, OP_DECODE = 0, 1, 2, 3, 4
OP_WINDOW_FORWARD, OP_WINDOW_BACKWARD, OP_WINDOW_DECODE = 5, 6, 7
OP_NORM_ROPE_BACKWARD, OP_NORM_ROPE_APPEND = 8, 9
OP_DECODE_Q4, OP_WINDOW_DECODE_Q4 = 10, 11
OP_PACKED_FORWARD, OP_PACKED_BACKWARD = 12, 13
ROPE_ROTATE, ROPE_CACHE, ROPE_CACHE_Q4, ROPE_PARTS, ROPE_AXES = 1, 2, 8, 8, 4
Q4_BLOCK_BYTES = 128 * 73  # 128 rows of a cache in 4 bits
STATUS_BITS = {1: "bad block index", 2: "work list overflow", 4: "device wait timeout",
               8: "internal layout check"}
_SYMBOLS = ("msa_workspace_size", "msa_forward", "msa_backward", "msa_warmup_forward",
            "msa_warmup_backward", "msa_device_status", "msa_status_string", "msa_last_error",
            "msa_profile_begin", "msa_profile_end", "msa_launch_count", "msa_forward_noalloc",
            "msa_forward_noalloc_status", "msa_selftest_wait_timeout", "msa_decode",
            "msa_window_workspace_size", "msa_window_wait_limit_ms", "msa_window_forward", "msa_window_backward",
            "msa_window_decode", "msa_norm_rope_forward", "msa_norm_rope_append",
            "msa_norm_rope_backward", "msa_norm_rope_workspace_size", "msa_norm_rope_axes_forward",
            "msa_norm_rope_axes_append", "msa_norm_rope_axes_backward", "msa_q4_cache_bytes",
            "msa_q4_read", "msa_window_decode_q4", "msa_decode_q4", "msa_packed_table_bytes",
            "msa_packed_plan", "msa_packed_workspace_size", "msa_packed_forward", "msa_packed_backward")


class MSAError(RuntimeError):
    pass


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("S", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("Hp", ctypes.c_int32), ("D", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("scale", ctypes.c_float)]


class WindowShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("S", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("window", ctypes.c_int32),
                ("sinks", ctypes.c_int32), ("scale", ctypes.c_float)]


class RopePart(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_batch", ctypes.c_int64), ("x_token", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("y_batch", ctypes.c_int64), ("y_token", ctypes.c_int64),
                ("dx", ctypes.c_void_p), ("dx_batch", ctypes.c_int64),
                ("dx_token", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("dweight", ctypes.c_void_p), ("heads", ctypes.c_int32), ("flags", ctypes.c_int32)]


class RopeShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("D", ctypes.c_int32),
                ("rotary", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("eps", ctypes.c_float)]


class PackedShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "Hq", "Hkv", "D", "window")]


class PackedCounts(ctypes.Structure):  # msa_packed_plan_t
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "tokens", "Hq", "Hkv", "window", "fwd_tiles", "fwd_units",
                                              "dq_units", "chunk", "items", "slots", "joins")]


class RopeAxes(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int32), ("of_pair", ctypes.c_uint8 * 64)]


_lib = None
_lock = threading.Lock()


def load_library(path: str = LIB_PATH):
    """Load libmsa.so (raises MSAError if it is missing: there is no CPU fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise MSAError(f"{path} not found: build it with block_sparse_attention_qp_gb300.build")
        lib = ctypes.CDLL(path)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        SP = ctypes.POINTER(Shape)
        lib.msa_workspace_size.argtypes = [SP, I]
        lib.msa_workspace_size.restype = Z
        lib.msa_forward.argtypes = [SP, P, P, P, P, P, P, I, P, P, P, Z, P]
        lib.msa_backward.argtypes = [SP, P, P, P, P, P, P, P, P, P, F, P, P, P, P, P, P, P, P, Z,
                                     P]
        lib.msa_warmup_forward.argtypes = [SP, P, P, P, P, P, P, Z, P]
        lib.msa_warmup_backward.argtypes = [SP, P, P, P, P, P, P, P, P, F, P, P, P, P, P, P, P, P,
                                            Z, P]
        lib.msa_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint), P]
        lib.msa_decode.argtypes = [SP, P, P, P, P, P, P, P, P, P, P, Z, P]
        lib.msa_decode.restype = I
        WP, RS = ctypes.POINTER(WindowShape), ctypes.POINTER(RopeShape)
        RP = P  # an array of RopePart, or its bytes
        lib.msa_window_workspace_size.argtypes = [WP, I]
        lib.msa_window_workspace_size.restype = Z
        lib.msa_window_wait_limit_ms.argtypes = [WP, I]
        lib.msa_window_wait_limit_ms.restype = ctypes.c_uint
        lib.msa_window_forward.argtypes = [WP, P, P, P, P, P, P, Z, P]
        lib.msa_window_backward.argtypes = [WP, P, P, P, P, P, P, P, P, P, P, Z, P]
        lib.msa_window_decode.argtypes = [WP, P, P, P, P, P, P, P, Z, P]
        lib.msa_norm_rope_forward.argtypes = [RS, RP, I, P, P, P]
        lib.msa_norm_rope_append.argtypes = [RS, RP, I, P, P, P, Z, P]
        lib.msa_norm_rope_backward.argtypes = [RS, RP, I, P, P, P, Z, P]
        lib.msa_norm_rope_workspace_size.argtypes = [I, I]
        lib.msa_norm_rope_workspace_size.restype = Z
        for name in ("msa_window_forward", "msa_window_backward", "msa_window_decode",
                     "msa_norm_rope_forward", "msa_norm_rope_append", "msa_norm_rope_backward"):
            getattr(lib, name).restype = I
        AP = ctypes.POINTER(RopeAxes)
        lib.msa_norm_rope_axes_forward.argtypes = [RS, RP, I, P, P, AP, P]
        lib.msa_norm_rope_axes_append.argtypes = [RS, RP, I, P, P, P, AP, P, Z, P]
        lib.msa_norm_rope_axes_backward.argtypes = [RS, RP, I, P, P, AP, P, Z, P]
        lib.msa_q4_cache_bytes.argtypes = [I, I, I]
        lib.msa_q4_cache_bytes.restype = Z
        lib.msa_q4_read.argtypes = [P, I, I, I, I, I, P, P]
        lib.msa_window_decode_q4.argtypes = [WP, P, P, P, P, P, P, P, Z, P]
        lib.msa_decode_q4.argtypes = [SP, P, P, P, P, P, P, P, P, P, P, Z, P]
        KP, LP, CP = ctypes.POINTER(PackedShape), ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(PackedCounts)
        lib.msa_packed_table_bytes.argtypes = [KP, LP, I]
        lib.msa_packed_table_bytes.restype = Z
        lib.msa_packed_plan.argtypes = [KP, LP, I, CP, P, Z, P]
        lib.msa_packed_workspace_size.argtypes = [CP, I]
        lib.msa_packed_workspace_size.restype = Z
        lib.msa_packed_forward.argtypes = [CP, P, Z, P, P, P, F, P, P, P, Z, P]
        lib.msa_packed_backward.argtypes = [CP, P, Z, P, P, P, P, P, P, F, P, P, P, P, Z, P]
        for name in ("msa_packed_plan", "msa_packed_forward", "msa_packed_backward"):
            getattr(lib, name).restype = I
        for name in ("msa_norm_rope_axes_forward", "msa_norm_rope_axes_append", "msa_norm_rope_axes_backward",
                     "msa_q4_read", "msa_window_decode_q4", "msa_decode_q4"):
            getattr(lib, name).restype = I
        lib.msa_status_string.argtypes = [I]
        lib.msa_status_string.restype = ctypes.c_char_p
        lib.msa_last_error.restype = ctypes.c_char_p
        for name in ("msa_forward", "msa_backward", "msa_warmup_forward", "msa_warmup_backward",
                     "msa_device_status", "msa_profile_begin", "msa_profile_end"):
            getattr(lib, name).restype = I
        lib.msa_profile_end.argtypes = [ctypes.c_char_p, Z]
        lib.msa_forward_noalloc.argtypes = [SP, P, P, P, P, P, P, I, P, P, P]
        lib.msa_forward_noalloc.restype = I
        lib.msa_forward_noalloc_status.argtypes = [ctypes.POINTER(ctypes.c_uint), P]
        lib.msa_forward_noalloc_status.restype = I
        lib.msa_launch_count.restype = ctypes.c_longlong
        lib.msa_selftest_wait_timeout.argtypes = [P, ctypes.c_uint, P]
        lib.msa_selftest_wait_timeout.restype = I
        _lib = lib
        return lib


def _check(rc: int, what: str):
    if rc != 0:
        lib = load_library()
        raise MSAError(f"{what}: {lib.msa_status_string(rc).decode()} "
                       f"({lib.msa_last_error().decode()})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _on_tensor_device(fn):
    """Runs fn with the CUDA device of its first tensor argument current, so that the library
    launches on the device that holds the data (with that device's current stream); every other
    tensor argument must be on the same device."""
    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        tensors = [a for a in list(args) + list(kwargs.values()) if isinstance(a, torch.Tensor)]
        if not tensors or not tensors[0].is_cuda:
            return fn(*args, **kwargs)
        dev = tensors[0].device
        for t in tensors[1:]:
            if t.device != dev:
                raise MSAError(f"{fn.__name__}: tensors on {dev} and {t.device}; all arguments "
                               "must be on one device")
        with torch.cuda.device(dev):
            return fn(*args, **kwargs)
    return wrapper


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _req(t, name, dtype=torch.bfloat16, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise MSAError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise MSAError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise MSAError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise MSAError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def make_shape(q, k, qp, top_k, scale) -> Shape:
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    Hp = qp.shape[2] if qp is not None else Hkv
    return Shape(B, S, Hq, Hkv, Hp, D, int(top_k), float(scale))


def msa_workspace_size(shape: Shape, op: int) -> int:
    n = load_library().msa_workspace_size(ctypes.byref(shape), op)
    if n == 0:
        raise MSAError(f"unsupported shape for op {op}: "
                       f"{load_library().msa_last_error().decode()}")
    return int(n)


def workspace(shape: Shape, op: int, device) -> torch.Tensor:
    """Fresh workspace (uint8 tensor, 256-byte aligned by the CUDA caching allocator)."""
    return torch.empty(msa_workspace_size(shape, op), dtype=torch.uint8, device=device)


_WS_CACHE: dict = {}


def cached_workspace(shape: Shape, op: int, device) -> torch.Tensor:
    """Workspace kept per (device, current stream) and reused by later calls on that stream: the
    stream orders each call after the previous one, and no call leaves state in it that a later
    call reads.  Grows (never shrinks) to the largest size asked for; clear_workspace_cache()
    releases it.  A call that is being captured gets memory of its graph's own instead: graphs captured on
    one stream may be replayed on several, and outlive the cache."""
    device = torch.device(device)
    with torch.cuda.device(device):
        if torch.cuda.is_current_stream_capturing():
            return workspace(shape, op, device)
    key = (device.index if device.index is not None else torch.cuda.current_device(),
           torch.cuda.current_stream(device).cuda_stream)
    need = msa_workspace_size(shape, op)
    ws = _WS_CACHE.get(key)
    if ws is None or ws.numel() < need:
        _WS_CACHE.pop(key, None)
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        _WS_CACHE[key] = ws
    return ws


def clear_workspace_cache() -> None:
    _WS_CACHE.clear()


def _kl_grad_args(kl_grad, device):
    """(host value, device pointer) for the library's kl_grad / kl_grad_dev pair: a number is
    passed by value; a one-element fp32 tensor on the device is read by the kernel, so the host
    never waits for it."""
    if isinstance(kl_grad, torch.Tensor):
        if kl_grad.numel() != 1:
            raise MSAError(f"kl_grad must have one element, got shape {tuple(kl_grad.shape)}")
        if kl_grad.device != torch.device(device):
            raise MSAError(f"kl_grad is on {kl_grad.device}, the inputs on {device}")
        t = kl_grad.detach().reshape(()).to(torch.float32).contiguous()
        return 0.0, t
    return float(kl_grad), None


@_on_tensor_device
def msa_device_status(ws: torch.Tensor) -> int:
    """Read and clear the device status word of a workspace (synchronises the stream)."""
    flags = ctypes.c_uint(0)
    _check(load_library().msa_device_status(_ptr(ws), ctypes.byref(flags), _stream(ws.device)),
           "msa_device_status")
    return int(flags.value)


@_on_tensor_device
def selftest_wait_timeout(ws: torch.Tensor, limit_us: int = 1000) -> None:
    """Run the library's bounded-wait self-test on ws's device (see msa_selftest_wait_timeout);
    the timeout shows up in msa_device_status(ws)."""
    _check(load_library().msa_selftest_wait_timeout(_ptr(ws), int(limit_us), _stream(ws.device)),
           "msa_selftest_wait_timeout")


def profile_begin() -> None:
    """Start per-kernel CUDA-event timing inside the library (measurement aid)."""
    _check(load_library().msa_profile_begin(), "msa_profile_begin")


def profile_end() -> dict:
    """Stop timing; returns {kernel name: (launches, total milliseconds)}."""
    buf = ctypes.create_string_buffer(1 << 16)
    _check(load_library().msa_profile_end(buf, len(buf)), "msa_profile_end")
    out = {}
    for line in buf.value.decode().splitlines():
        name, n, ms = line.split()
        out[name] = (int(n), float(ms))
    return out


def launch_count() -> int:
    """Kernels launched by the library since it was loaded."""
    return int(load_library().msa_launch_count())


@_on_tensor_device
def msa_forward(q, k, v, qp, kp, top_k: int, scale: float, block_idx=None, ws=None):
    """Sparse forward.  Returns (o, lse, block_idx).  block_idx given -> used as the selection."""
    B, S, Hq, D = q.shape
    Hkv, Hp = k.shape[2], qp.shape[2]
    for t, n, shp in ((q, "q", None), (k, "k", (B, S, Hkv, D)), (v, "v", (B, S, Hkv, D)),
                      (qp, "qp", (B, S, Hp, D)), (kp, "kp", (B, S, 1, D))):
        _req(t, n, shape=shp)
    shape = make_shape(q, k, qp, top_k, scale)
    given = block_idx is not None
    if given:
        _req(block_idx, "block_idx", torch.int32, (B, Hp, S, top_k))
    else:
        block_idx = torch.empty((B, Hp, S, top_k), dtype=torch.int32, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(shape, OP_FORWARD, q.device)
    _check(load_library().msa_forward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(qp),
                                      _ptr(kp), _ptr(block_idx), int(given), _ptr(o), _ptr(lse),
                                      _ptr(ws), ws.numel(), _stream(q.device)), "msa_forward")
    return o, lse, block_idx


@_on_tensor_device
def msa_forward_noalloc(q, k, v, qp, kp, top_k: int, scale: float, block_idx=None):
    """msa_forward without a workspace: the library's fixed device scratch array is used instead
    (see include/msa.h).  Returns (o, lse, block_idx)."""
    B, S, Hq, D = q.shape
    Hp = qp.shape[2]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (qp, "qp"), (kp, "kp")):
        _req(t, n)
    shape = make_shape(q, k, qp, top_k, scale)
    given = block_idx is not None
    if given:
        _req(block_idx, "block_idx", torch.int32, (B, Hp, S, top_k))
    else:
        block_idx = torch.empty((B, Hp, S, top_k), dtype=torch.int32, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    _check(load_library().msa_forward_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                              _ptr(qp), _ptr(kp), _ptr(block_idx), int(given),
                                              _ptr(o), _ptr(lse), _stream(q.device)),
           "msa_forward_noalloc")
    return o, lse, block_idx


def msa_forward_noalloc_status(device=None) -> int:
    """Read and clear the status word of the fixed scratch array msa_forward_noalloc uses on the
    current device (synchronises the current stream)."""
    flags = ctypes.c_uint(0)
    _check(load_library().msa_forward_noalloc_status(ctypes.byref(flags), _stream(device)),
           "msa_forward_noalloc_status")
    return int(flags.value)


@_on_tensor_device
def msa_backward(q, k, v, qp, kp, o, lse, dout, block_idx, top_k: int, scale: float,
                 kl_grad=1.0, ws=None, return_kl: bool = False):
    """Sparse backward.  Returns (dq, dk, dv, dqp, dkp), plus the KL value L_KL as a 0-d fp32
    CUDA tensor when return_kl (computed on the device; no host synchronisation).  kl_grad: a
    number, or a one-element tensor on the device (read by the kernel)."""
    B, S, Hq, D = q.shape
    Hp = qp.shape[2]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (qp, "qp"), (kp, "kp"), (o, "o"), (dout, "dout")):
        _req(t, n)
    _req(lse, "lse", torch.float32, (B, Hq, S))
    _req(block_idx, "block_idx", torch.int32, (B, Hp, S, top_k))
    shape = make_shape(q, k, qp, top_k, scale)
    grads = [torch.empty_like(x) for x in (q, k, v, qp, kp)]
    kl = torch.empty((), dtype=torch.float32, device=q.device) if return_kl else None
    klg, klg_dev = _kl_grad_args(kl_grad, q.device)
    if ws is None:
        ws = workspace(shape, OP_BACKWARD, q.device)
    _check(load_library().msa_backward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(qp),
                                       _ptr(kp), _ptr(o), _ptr(lse), _ptr(dout), _ptr(block_idx),
                                       klg, _ptr(klg_dev), *map(_ptr, grads), _ptr(kl), _ptr(ws),
                                       ws.numel(), _stream(q.device)), "msa_backward")
    return tuple(grads) + ((kl,) if return_kl else ())


@_on_tensor_device
def msa_decode(q, qp, k_cache, v_cache, kp_cache, seq_len, top_k: int, scale: float, ws=None):
    """Decode step: q [B, Hq, D], qp [B, Hp, D] (the new tokens), caches k/v [B, S, Hkv, D] and
    kp [B, S, 1, D] (or [B, S, D]) already holding the new tokens at seq_len - 1, seq_len [B] int32
    on the device.  Returns (o [B, Hq, D], lse [B, Hq], block_idx [B, Hp, top_k])."""
    B, Hq, D = q.shape
    S, Hkv = k_cache.shape[1], k_cache.shape[2]
    Hp = qp.shape[1]
    for t, n in ((q, "q"), (qp, "qp"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                 (kp_cache, "kp_cache")):
        _req(t, n)
    _req(seq_len, "seq_len", torch.int32, (B,))
    shape = Shape(B, S, Hq, Hkv, Hp, D, int(top_k), float(scale))
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    idx = torch.empty((B, Hp, top_k), dtype=torch.int32, device=q.device)
    if ws is None:
        ws = workspace(shape, OP_DECODE, q.device)
    _check(load_library().msa_decode(ctypes.byref(shape), _ptr(q), _ptr(qp), _ptr(k_cache),
                                     _ptr(v_cache), _ptr(kp_cache), _ptr(seq_len), _ptr(idx),
                                     _ptr(o), _ptr(lse), _ptr(ws), ws.numel(), _stream(q.device)),
           "msa_decode")
    return o, lse, idx


@_on_tensor_device
def msa_warmup_forward(q, k, v, scale: float, ws=None):
    """Dense causal forward (warmup).  Returns (o, lse)."""
    B, S, Hq, D = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _req(t, n)
    shape = make_shape(q, k, None, 0, scale)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(shape, OP_WARMUP_FORWARD, q.device)
    _check(load_library().msa_warmup_forward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                             _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
                                             _stream(q.device)), "msa_warmup_forward")
    return o, lse


@_on_tensor_device
def msa_warmup_backward(q, k, v, qp, kp, o, lse, dout, scale: float, kl_grad=1.0,
                        ws=None, return_kl: bool = False):
    """Dense warmup backward (proxy KL over the full causal prefix).  Returns grads (and the KL
    value as a 0-d fp32 CUDA tensor when return_kl).  kl_grad as in msa_backward."""
    B, S, Hq, D = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (qp, "qp"), (kp, "kp"), (o, "o"), (dout, "dout")):
        _req(t, n)
    _req(lse, "lse", torch.float32, (B, Hq, S))
    shape = make_shape(q, k, qp, 0, scale)
    grads = [torch.empty_like(x) for x in (q, k, v, qp, kp)]
    kl = torch.empty((), dtype=torch.float32, device=q.device) if return_kl else None
    klg, klg_dev = _kl_grad_args(kl_grad, q.device)
    if ws is None:
        ws = workspace(shape, OP_WARMUP_BACKWARD, q.device)
    _check(load_library().msa_warmup_backward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                              _ptr(qp), _ptr(kp), _ptr(o), _ptr(lse), _ptr(dout),
                                              klg, _ptr(klg_dev), *map(_ptr, grads), _ptr(kl),
                                              _ptr(ws), ws.numel(), _stream(q.device)),
           "msa_warmup_backward")
    return tuple(grads) + ((kl,) if return_kl else ())


class _MSAFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, qp, kp, q, k, v, top_k, scale, warmup):
        qp, kp, q, k, v = (x.contiguous() for x in (qp, kp, q, k, v))
        if warmup:
            o, lse = msa_warmup_forward(
                q, k, v, scale,
                ws=cached_workspace(make_shape(q, k, None, 0, scale), OP_WARMUP_FORWARD, q.device))
            idx = None
        else:
            o, lse, idx = msa_forward(
                q, k, v, qp, kp, top_k, scale,
                ws=cached_workspace(make_shape(q, k, qp, top_k, scale), OP_FORWARD, q.device))
        ctx.save_for_backward(qp, kp, q, k, v, o, lse, *(() if idx is None else (idx,)))
        ctx.top_k, ctx.scale, ctx.warmup = top_k, scale, warmup
        kl = torch.zeros((), dtype=torch.float32, device=q.device)
        return o, kl

    @staticmethod
    def backward(ctx, do, dkl):
        saved = ctx.saved_tensors
        qp, kp, q, k, v, o, lse = saved[:7]
        kl_grad = 0.0 if dkl is None else dkl  # a device tensor: read by the kernel, no sync
        do = torch.zeros_like(o) if do is None else do.contiguous()
        if ctx.warmup:
            ws = cached_workspace(make_shape(q, k, qp, 0, ctx.scale), OP_WARMUP_BACKWARD, q.device)
            dq, dk, dv, dqp, dkp = msa_warmup_backward(q, k, v, qp, kp, o, lse, do, ctx.scale,
                                                       kl_grad, ws=ws)
        else:
            ws = cached_workspace(make_shape(q, k, qp, ctx.top_k, ctx.scale), OP_BACKWARD,
                                  q.device)
            dq, dk, dv, dqp, dkp = msa_backward(q, k, v, qp, kp, o, lse, do, saved[7], ctx.top_k,
                                                ctx.scale, kl_grad, ws=ws)
        return dqp, dkp, dq, dk, dv, None, None, None


def msa_func(Q_proxy, K_proxy, Q, K, V, top_k: int, scale: float):
    """Sparse MSA attention with the Flash-MSA call convention.  Returns (attn_out, kl_loss);
    add kl_loss to the training loss so that backward() trains the proxy heads."""
    return _MSAFunction.apply(Q_proxy, K_proxy, Q, K, V, int(top_k), float(scale), False)


def msa_warmup_func(Q_proxy, K_proxy, Q, K, V, top_k: int, scale: float):
    """Warmup mode: dense main attention, proxy trained over the full causal prefix."""
    return _MSAFunction.apply(Q_proxy, K_proxy, Q, K, V, int(top_k), float(scale), True)


# ---------------------------------------------------------------- sliding-window attention
# The entry points below serve single tokens too, where the host's part of a call counts: arguments are
# looked at once by a fast test, and only a failing one is taken apart for its message.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


class _Guard:
    """Makes a device current for a block (torch.cuda.device costs microseconds even where it is).  Entered with a CUDA
    tensor at hand, so CUDA is up."""
    __slots__ = ("device", "entered")

    def __init__(self, device):
        self.device = device

    def __enter__(self):
        self.entered = None
        if _current_device() != self.device.index:
            self.entered = torch.cuda.device(self.device)
            self.entered.__enter__()

    def __exit__(self, *exc):
        if self.entered is not None:
            self.entered.__exit__(*exc)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device) -> int:
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _ask(t, name, dtype, shape, device):
    """t is a contiguous CUDA tensor of this type, shape and device; returns its address."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device \
            and t.is_contiguous():
        return t.data_ptr()
    _req(t, name, dtype, shape)
    raise MSAError(f"{name} is on {t.device}, the first argument on {device}")


def _dims(t, name, n):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dim() != n:
        raise MSAError(f"{name} has shape {tuple(t.shape)}, expected {n} dimensions")
    return t.shape


def make_window_shape(q, k, window, sinks, scale) -> WindowShape:
    """Shape of a window op: q [B, S, Hq, D] (decode: [B, Hq, D]), k [B, S, Hkv, D]."""
    B, S, Hkv = k.shape[:3]
    return WindowShape(B, S, q.shape[-2], Hkv, q.shape[-1], _int32(window, "window"),
                       _int32(sinks, "sinks"), float(scale))


def _int32(x, name) -> int:
    """x as an int32; larger values (a window of "everything") saturate."""
    x = int(x)
    if x < -2 ** 31:
        raise MSAError(f"{name} is out of range: {x}")
    return min(x, 2 ** 31 - 1)


def _whole(x, name) -> int:
    """x as an int, without dropping a fraction."""
    try:
        n = int(x)
    except (TypeError, ValueError, OverflowError):  # nan, inf, no number
        n = None
    if n is None or n != x:
        raise MSAError(f"{name} must be whole numbers, got {x}")
    return n


@functools.lru_cache(maxsize=4096)
def _window_bytes(op, *shape):
    lib = load_library()
    n = int(lib.msa_window_workspace_size(ctypes.byref(WindowShape(*shape)), op))
    if n == 0:
        raise MSAError(f"unsupported shape for op {op}: {lib.msa_last_error().decode()}")
    return n


@functools.lru_cache(maxsize=4096)
def _window_call(op, *shape):
    """(the shape as an argument of the library, bytes of workspace); nothing writes to the shape."""
    return ctypes.byref(WindowShape(*shape)), _window_bytes(op, *shape)


def msa_window_workspace_size(shape: WindowShape, op: int) -> int:
    return _window_bytes(op, shape.B, shape.S, shape.Hq, shape.Hkv, shape.D, shape.window, shape.sinks,
                         shape.scale)


def msa_window_wait_limit_ms(shape: WindowShape, op: int) -> int:
    """The longest that a wait inside the op's kernels may last before the call ends with the timeout bit in
    msa_device_status(ws)."""
    lib = load_library()
    ms = int(lib.msa_window_wait_limit_ms(ctypes.byref(shape), op))
    if ms == 0:
        raise MSAError(f"unsupported shape for op {op}: {lib.msa_last_error().decode()}")
    return ms


def window_workspace(shape: WindowShape, op: int, device) -> torch.Tensor:
    """Fresh workspace of a window op (uint8 tensor)."""
    return torch.empty(msa_window_workspace_size(shape, op), dtype=torch.uint8, device=device)


def _ws(ws, need, device):
    """(address, bytes, tensor) of the caller's workspace, or of a fresh one of `need` bytes."""
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _req(ws, "ws", torch.uint8)
        if ws.device != device:
            raise MSAError(f"ws is on {ws.device}, the inputs on {device}")
    return ws.data_ptr(), ws.numel(), ws


def _window_args(q, k, v, window, sinks, scale, op, ws, dims):
    """Checks q, k and v; returns (device, addresses, shape, workspace)."""
    qs = _dims(q, "q", dims)
    nk, nv = ("k", "v") if dims == 4 else ("k_cache", "v_cache")
    B, S, Hkv, _ = _dims(k, nk, 4)
    Hq, D = qs[-2:]
    dev = q.device
    if not q.is_cuda:
        raise MSAError("q must be a CUDA tensor")
    kv = (B, S, Hkv, D)
    ptrs = (_ask(q, "q", torch.bfloat16, (B, S, Hq, D) if dims == 4 else (B, Hq, D), dev),
            _ask(k, nk, torch.bfloat16, kv, dev), _ask(v, nv, torch.bfloat16, kv, dev))
    window, sinks, scale = _int32(window, "window"), _int32(sinks, "sinks"), float(scale)
    need = _window_bytes(op, B, S, Hq, Hkv, D, window, sinks, scale) if ws is None else 0
    return dev, ptrs, WindowShape(B, S, Hq, Hkv, D, window, sinks, scale), need


def msa_window_forward(q, k, v, window: int, sinks: int, scale: float, ws=None):
    """Causal GQA attention of every query over the last ``window`` tokens (itself included) and the
    first ``sinks`` tokens.  q [B, S, Hq, 128], k, v [B, S, Hkv, 128], any S.  Returns (o, lse).  Rows that a
    query does not see never reach it, whatever they hold (padding behind a ragged prompt may be uninitialised)."""
    dev, ptrs, shape, need = _window_args(q, k, v, window, sinks, scale, OP_WINDOW_FORWARD, ws, 4)
    with _Guard(dev):
        wp, wn, ws = _ws(ws, need, dev)
        o = torch.empty_like(q)
        lse = torch.empty((shape.B, shape.Hq, shape.S), dtype=torch.float32, device=dev)
        rc = load_library().msa_window_forward(ctypes.byref(shape), *ptrs, o.data_ptr(), lse.data_ptr(),
                                               wp, wn, _stream_of(dev))
    if rc:
        _check(rc, "msa_window_forward")
    return o, lse


def msa_window_backward(q, k, v, o, lse, dout, window: int, sinks: int, scale: float, ws=None):
    """Gradients (dq, dk, dv) of sum(o * dout); o, lse from msa_window_forward on the same inputs, which must all be
    finite, padding included."""
    dev, ptrs, shape, need = _window_args(q, k, v, window, sinks, scale, OP_WINDOW_BACKWARD, ws, 4)
    op = _ask(o, "o", torch.bfloat16, q.shape, dev)
    lp = _ask(lse, "lse", torch.float32, (shape.B, shape.Hq, shape.S), dev)
    dp = _ask(dout, "dout", torch.bfloat16, q.shape, dev)
    with _Guard(dev):
        wp, wn, ws = _ws(ws, need, dev)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        rc = load_library().msa_window_backward(ctypes.byref(shape), *ptrs, op, lp, dp, dq.data_ptr(),
                                                dk.data_ptr(), dv.data_ptr(), wp, wn, _stream_of(dev))
    if rc:
        _check(rc, "msa_window_backward")
    return dq, dk, dv


def msa_window_decode(q, k_cache, v_cache, seq_len, window: int, sinks: int, scale: float, ws=None):
    """Decode step: q [B, Hq, 128] against caches [B, S, Hkv, 128] that already hold the new tokens at
    seq_len - 1 (seq_len [B] int32 on the device).  Returns (o [B, Hq, 128], lse [B, Hq]); the rows of
    a sequence whose length is not in 1 .. S are not written (msa_device_status tells)."""
    dev, ptrs, shape, need = _window_args(q, k_cache, v_cache, window, sinks, scale, OP_WINDOW_DECODE,
                                          ws, 3)
    sp = _ask(seq_len, "seq_len", torch.int32, (shape.B,), dev)
    with _Guard(dev):
        wp, wn, ws = _ws(ws, need, dev)
        o = torch.empty_like(q)
        lse = torch.empty((shape.B, shape.Hq), dtype=torch.float32, device=dev)
        rc = load_library().msa_window_decode(ctypes.byref(shape), *ptrs, sp, o.data_ptr(),
                                              lse.data_ptr(), wp, wn, _stream_of(dev))
    if rc:
        _check(rc, "msa_window_decode")
    return o, lse


class _WindowFunction(torch.autograd.Function):
    # Workspaces are allocated per call: the caching allocator hands a captured graph memory of its
    # own, so graphs captured on one stream never share one.
    @staticmethod
    def forward(ctx, q, k, v, window, sinks, scale):
        q, k, v = (x.contiguous() for x in (q, k, v))
        o, lse = msa_window_forward(q, k, v, window, sinks, scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.how = (window, sinks, scale)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        return msa_window_backward(q, k, v, o, lse, do.contiguous(), *ctx.how) + (None,) * 3


def msa_window_func(Q, K, V, window: int, sinks: int, scale: float):
    """Sliding-window attention with autograd (msa_window_forward / msa_window_backward); returns
    attn_out.  To be trained through, Q, K, V and the gradient have to be finite, padding included."""
    return _WindowFunction.apply(Q, K, V, int(window), int(sinks), float(scale))


# ---------------------------------------------------------------- attention over packed sequences
class PackedPlan:
    """What msa_packed_plan returns: the lengths' tables on the device, for the calls of one step (any number of
    layers) over tensors of ``rows`` rows.  Made in the order of the stream that was current: calls on another one have to
    wait for it (an event).  The tables outlive the plan until the calls that use them are done, on whatever stream."""
    __slots__ = ("counts", "table", "rows", "tokens", "Hq", "Hkv", "device", "_bytes", "_stream")

    def __init__(self, counts, table, stream):
        self.counts, self.table, self.device, self._stream = counts, table, table.device, stream
        self.rows, self.tokens, self.Hq, self.Hkv = counts.rows, counts.tokens, counts.Hq, counts.Hkv
        self._bytes = {}

    def used_on(self, stream: int) -> None:
        """Called for every stream that reads the table: dropped, it goes back to its own stream's memory, which another
        stream's kernels may still be reading."""
        if stream != self._stream:
            self.table.record_stream(torch.cuda.current_stream(self.device))

    def workspace_size(self, op: int) -> int:
        n = self._bytes.get(op)
        if n is None:
            lib = load_library()
            n = self._bytes[op] = int(lib.msa_packed_workspace_size(ctypes.byref(self.counts), op))
            if n == 0:
                raise MSAError(f"op {op}: {lib.msa_last_error().decode()}")
        return n


def msa_packed_plan(lengths, heads: int, kv_heads: int, rows: int | None = None, window: int | None = None,
                    device=None) -> PackedPlan:
    """Plan of sequences of these lengths (numbers on the host, zeros among them) that lie one behind the other in
    tensors of ``rows`` rows (default: their sum), each token seeing the tokens before it of its own sequence and,
    with a window, the last ``window`` of them.  Neither copies from the host nor waits."""
    if isinstance(lengths, torch.Tensor):
        if lengths.is_cuda:
            raise MSAError("lengths must be on the host (a plan does not wait for the device)")
        lengths = lengths.tolist()
    lengths = list(lengths)
    try:  # (0.04 us a sequence on the host, converted one by one 0.16)
        lengths = array.array("i", lengths)
    except (TypeError, OverflowError):
        lengths = [_whole(n, "lengths") for n in lengths]
        if not 0 <= min(lengths) <= max(lengths) < 2 ** 31:
            raise MSAError("lengths must be in 0 .. 2^31 - 1") from None
        lengths = array.array("i", lengths)
    if lengths and min(lengths) < 0:
        raise MSAError("lengths must be in 0 .. 2^31 - 1")
    total = sum(lengths)
    rows = total if rows is None else _whole(rows, "rows")
    if not total <= rows < 2 ** 31:
        raise MSAError(f"{total} tokens in {rows} rows")
    n = len(lengths)
    arr = (ctypes.c_int32 * n).from_buffer(lengths) if n else (ctypes.c_int32 * 1)()
    shape = PackedShape(rows, _int32(_whole(heads, "heads"), "heads"), _int32(_whole(kv_heads, "kv_heads"), "kv_heads"), 128,
                        rows if window is None else _int32(window, "window"))
    dev = torch.device("cuda" if device is None else device)
    if dev.type != "cuda":
        raise MSAError(f"device must be a CUDA device, got {dev}")
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    lib = load_library()
    with _Guard(dev):
        need = int(lib.msa_packed_table_bytes(ctypes.byref(shape), arr, n))
        if need == 0:
            raise MSAError(f"msa_packed_plan: {lib.msa_last_error().decode()}")
        table, counts, stream = torch.empty(need, dtype=torch.uint8, device=dev), PackedCounts(), _stream_of(dev)
        rc = lib.msa_packed_plan(ctypes.byref(shape), arr, n, ctypes.byref(counts), table.data_ptr(), need, stream)
    if rc:
        _check(rc, "msa_packed_plan")
    return PackedPlan(counts, table, stream)


def _packed_args(q, k, v, plan):
    """Checks q, k and v against the plan; returns their addresses."""
    if not isinstance(plan, PackedPlan):
        raise TypeError("plan must be a PackedPlan (msa_packed_plan)")
    _dims(q, "q", 3)
    if not q.is_cuda:
        raise MSAError("q must be a CUDA tensor")
    dev = plan.device
    if q.device != dev:
        raise MSAError(f"q is on {q.device}, the plan on {dev}")
    kv = (plan.rows, plan.Hkv, 128)
    return (_ask(q, "q", torch.bfloat16, (plan.rows, plan.Hq, 128), dev), _ask(k, "k", torch.bfloat16, kv, dev),
            _ask(v, "v", torch.bfloat16, kv, dev))


def msa_packed_forward(q, k, v, plan: PackedPlan, scale: float, ws=None):
    """Causal GQA attention over packed sequences: q [rows, Hq, 128], k, v [rows, Hkv, 128].  Returns (o, lse
    [Hq, rows]); rows behind the last sequence are 0 and -inf whatever the inputs hold there."""
    ptrs = _packed_args(q, k, v, plan)
    dev = plan.device
    with _Guard(dev):
        wp, wn, ws = _ws(ws, plan.workspace_size(OP_PACKED_FORWARD) if ws is None else 0, dev)
        o = torch.empty_like(q)
        lse = torch.empty((plan.Hq, plan.rows), dtype=torch.float32, device=dev)
        stream = _stream_of(dev)
        plan.used_on(stream)
        rc = load_library().msa_packed_forward(ctypes.byref(plan.counts), plan.table.data_ptr(), plan.table.numel(), *ptrs,
                                               float(scale), o.data_ptr(), lse.data_ptr(), wp, wn, stream)
    if rc:
        _check(rc, "msa_packed_forward")
    return o, lse


def msa_packed_backward(q, k, v, o, lse, dout, plan: PackedPlan, scale: float, ws=None):
    """Gradients (dq, dk, dv) of sum(o * dout); o, lse from msa_packed_forward on the same inputs, whose rows of the
    sequences must be finite.  Rows behind the last sequence are 0 whatever the inputs hold there."""
    ptrs = _packed_args(q, k, v, plan)
    dev = plan.device
    op = _ask(o, "o", torch.bfloat16, q.shape, dev)
    lp = _ask(lse, "lse", torch.float32, (plan.Hq, plan.rows), dev)
    dp = _ask(dout, "dout", torch.bfloat16, q.shape, dev)
    with _Guard(dev):
        wp, wn, ws = _ws(ws, plan.workspace_size(OP_PACKED_BACKWARD) if ws is None else 0, dev)
        grads = dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        stream = _stream_of(dev)
        plan.used_on(stream)
        rc = load_library().msa_packed_backward(ctypes.byref(plan.counts), plan.table.data_ptr(), plan.table.numel(), *ptrs, op,
                                                lp, dp, float(scale), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), wp, wn,
                                                stream)
    if rc:
        _check(rc, "msa_packed_backward")
    return grads


class _PackedFunction(torch.autograd.Function):
    # (workspaces per call, as in _WindowFunction)
    @staticmethod
    def forward(ctx, q, k, v, plan, scale):
        q, k, v = (x.contiguous() for x in (q, k, v))
        o, lse = msa_packed_forward(q, k, v, plan, scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.how = (plan, scale)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        return msa_packed_backward(q, k, v, o, lse, do.contiguous(), *ctx.how) + (None,) * 2


def msa_packed_func(Q, K, V, plan: PackedPlan, scale: float):
    """Attention over packed sequences with autograd; returns attn_out."""
    return _PackedFunction.apply(Q, K, V, plan, float(scale))


# ---------------------------------------------------------------- norm and rotation of the heads
_PART = struct.Struct("@NqqNqqNqqNNii")  # RopePart
assert _PART.size == ctypes.sizeof(RopePart)


def _rows(t, name, B=None, N=None, H=None, write=False):
    """Checks a part tensor [B, N, H, 128]: rows contiguous, heads 128 apart, batch and token strides
    free.  Returns its (pointer, batch stride, token stride)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    shape = t.shape
    if t.dtype is not torch.bfloat16 or len(shape) != 4 or shape[3] != 128 or not t.is_cuda:
        if not t.is_cuda:
            raise MSAError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16:
            raise MSAError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
        raise MSAError(f"{name} has shape {tuple(shape)}, expected [B, N, heads, 128]")
    b, n, h, _ = shape
    if not (b and n and h) or (B is not None and B != b) or (N is not None and N != n) or (H is not None and H != h):
        raise MSAError(f"{name} has shape {tuple(shape)}, expected {(B, N, H, 128)}")
    sb, st, sh, sd = t.stride()
    if sd != 1 or (h > 1 and sh != 128):
        raise MSAError(f"{name}: rows must be contiguous and heads 128 elements apart "
                       f"(strides {t.stride()})")
    if b == 1:
        sb = 0
    if n == 1:
        st = 0
    ptr = t.data_ptr()
    if sb % 8 or st % 8 or ptr % 16:
        raise MSAError(f"{name} must be 16-byte aligned, batch and token strides multiples of 8")
    if write and (st != h * 128 or sb != n * st):
        need = h * 128  # a token's rows; no two tokens may share memory
        for stride, count in sorted(((sb, b), (st, n))):
            if count > 1:
                if stride < need:
                    raise MSAError(f"{name} overlaps itself (strides {t.stride()})")
                need += stride * (count - 1)
    return ptr, sb, st


_X_NAMES = [f"xs[{i}]" for i in range(ROPE_PARTS)]
_W_NAMES = [f"weights[{i}]" for i in range(ROPE_PARTS)]
_DY_NAMES = [f"dys[{i}]" for i in range(ROPE_PARTS)]
_DX_NAMES = [f"dxs[{i}]" for i in range(ROPE_PARTS)]
_C_NAMES = [f"caches[{i}]" for i in range(ROPE_PARTS)]


def _device_of(xs):
    if not xs or not isinstance(xs[0], torch.Tensor):
        raise TypeError("xs must be a sequence of tensors")
    if not xs[0].is_cuda:
        raise MSAError("xs[0] must be a CUDA tensor")
    return xs[0].device


def _on(t, name, device):
    if t.device != device:
        raise MSAError(f"{name} is on {t.device}, the inputs on {device}")


@functools.lru_cache(maxsize=64)
def _axes(axes, pairs):
    """The library's form of the axis of each pair."""
    if len(axes) != pairs:
        raise MSAError(f"axes has {len(axes)} entries, one for each of the {pairs} pairs expected")
    count = max(axes, default=0) + 1
    if min(axes, default=0) < 0 or count > ROPE_AXES:
        raise MSAError(f"axes must be 0 .. {ROPE_AXES - 1}, got {min(axes)} .. {count - 1}")
    return RopeAxes(count, (ctypes.c_uint8 * 64)(*axes))


def _rope_args(xs, weights, rotate, inv_freq, interleaved, eps, positions, dev, axes=None):
    """Checks what the norm and rotation entry points share; returns (shape, parts, inv_freq's and
    positions' addresses, the axes), a part being (x's pointer and strides, weight's address, heads, flags)."""
    count = len(xs)
    if not 1 <= count <= ROPE_PARTS:
        raise MSAError(f"between 1 and {ROPE_PARTS} tensors, got {count}")
    weights = [None] * count if weights is None else weights
    rotate = [inv_freq is not None] * count if rotate is None else rotate
    if len(weights) != count or len(rotate) != count:
        raise MSAError(f"{count} tensors, {len(weights)} weights, {len(rotate)} rotate flags")
    B, N = (xs[0].shape[0], xs[0].shape[1]) if xs[0].dim() == 4 else (None, None)
    parts = []
    for x, w, turn, nx, nw in zip(xs, weights, rotate, _X_NAMES, _W_NAMES):
        at = _rows(x, nx, B, N)
        if x.device != dev:
            _on(x, nx, dev)
        parts.append((at, 0 if w is None else _ask(w, nw, torch.float32, (128,), dev), x.shape[2],
                      ROPE_ROTATE if turn else 0))
    rotary, fp, pp = 0, None, None
    if inv_freq is not None:
        fp = _ask(inv_freq, "inv_freq", torch.float32, tuple(_dims(inv_freq, "inv_freq", 1)), dev)
        rotary = 2 * inv_freq.shape[0]
    elif any(rotate):
        raise MSAError("inv_freq is needed to rotate")
    if axes is not None:
        axes = _axes(tuple(axes), rotary // 2)
        if positions is None:
            raise MSAError("axes need positions")
        # more axes than the pairs use may be there
        A = _dims(positions, "positions", 3)[0]
        pp = _ask(positions, "positions", torch.int32, (max(A, axes.count), B, N), dev)
    elif positions is not None:
        pp = _ask(positions, "positions", torch.int32, (B, N), dev)
    return RopeShape(B, N, 128, rotary, 1 if interleaved else 0, 0, eps), parts, fp, pp, axes


@functools.lru_cache(maxsize=64)
def _rope_bytes(nparts, op):
    return int(load_library().msa_norm_rope_workspace_size(nparts, op))


def msa_norm_rope_forward(xs, weights, inv_freq, positions=None, eps: float = 1e-6, rotate=None,
                          interleaved: bool = False, axes=None):
    """RMS norm of every head's row and the position rotation, in one pass over several tensors.

    xs: up to 8 tensors [B, N, heads, 128] bf16 -- q, k, the proxy heads -- usually the slices of one
    packed projection (``packed.split(heads, 2)``; only rows and heads have to be dense).
    weights: one fp32 [128] or None (not normed) per tensor.  inv_freq: fp32 [rotary / 2], the first
    ``rotary`` (a multiple of 16) elements of a row turn by position * inv_freq; None: no rotation.
    rotate: one truth value per tensor (default: all).  positions: int32 [B, N], default 0 .. N - 1.
    axes: the axis (0 .. 3) of each of the rotary / 2 pairs, positions then int32 [axes, B, N] -- time, height
    and width of images and video: pair i turns by positions[axes[i]] * inv_freq[i].
    A tensor without weight and rotation is copied.  Returns contiguous tensors [B, N, heads, 128]."""
    dev = _device_of(xs)
    shape, parts, fp, pp, axes = _rope_args(xs, weights, rotate, inv_freq, interleaved, eps, positions, dev, axes)
    B, N, pack = shape.B, shape.N, _PART.pack
    with _Guard(dev):
        ys, rows = [], []
        for (px, sb, st), w, h, f in parts:
            y = torch.empty((B, N, h, 128), dtype=torch.bfloat16, device=dev)
            ys.append(y)
            rows.append(pack(px, sb, st, y.data_ptr(), N * h * 128, h * 128, 0, 0, 0, w, 0, h, f))
        packed = b"".join(rows)
        if axes is None:
            rc = load_library().msa_norm_rope_forward(ctypes.byref(shape), packed, len(ys), pp, fp,
                                                      _stream_of(dev))
        else:
            rc = load_library().msa_norm_rope_axes_forward(ctypes.byref(shape), packed, len(ys), pp, fp,
                                                           ctypes.byref(axes), _stream_of(dev))
    if rc:
        _check(rc, "msa_norm_rope_forward")
    return tuple(ys)


def msa_norm_rope_backward(xs, weights, dys, inv_freq, positions=None, eps: float = 1e-6,
                           rotate=None, interleaved: bool = False, dxs=None, ws=None, axes=None):
    """Gradients of msa_norm_rope_forward: (dxs, dweights), dweights fp32 [128] or None per tensor.
    dxs: where to write them (e.g. the slices of one packed gradient, or the dys), default new
    tensors; each may be its own part's x or dy, but overlap no other tensor of the call."""
    dev = _device_of(xs)
    shape, parts, fp, pp, axes = _rope_args(xs, weights, rotate, inv_freq, interleaved, eps, positions, dev, axes)
    n = len(xs)
    if len(dys) != n or (dxs is not None and len(dxs) != n):
        raise MSAError("one dy (and dx, where given) per tensor")
    with _Guard(dev):
        # one tensor for the weights' gradients: a row each
        dws = torch.empty((n, 128), dtype=torch.float32, device=dev)
        out_w, rows, dw = list(dws.unbind(0)), [], dws.data_ptr()
        B, N, pack, out_x = shape.B, shape.N, _PART.pack, [] if dxs is None else dxs
        for i, (at, w, h, f) in enumerate(parts):
            dy = dys[i]
            pdy = _rows(dy, _DY_NAMES[i], B, N, h)
            if dxs is None:
                dx = torch.empty((B, N, h, 128), dtype=torch.bfloat16, device=dev)
                out_x.append(dx)
                pdx = (dx.data_ptr(), N * h * 128, h * 128)
            else:
                dx = dxs[i]
                pdx = _rows(dx, _DX_NAMES[i], B, N, h, True)
            if dy.device != dev or dx.device != dev:
                _on(dy, _DY_NAMES[i], dev)
                _on(dx, _DX_NAMES[i], dev)
            rows.append(pack(*at, *pdy, *pdx, w, dw + 512 * i if w else 0, h, f))
            if not w:
                out_w[i] = None
        wp, wn, ws = _ws(ws, _rope_bytes(n, OP_NORM_ROPE_BACKWARD), dev)
        if axes is None:
            rc = load_library().msa_norm_rope_backward(ctypes.byref(shape), b"".join(rows), n, pp, fp, wp,
                                                       wn, _stream_of(dev))
        else:
            rc = load_library().msa_norm_rope_axes_backward(ctypes.byref(shape), b"".join(rows), n, pp, fp,
                                                            ctypes.byref(axes), wp, wn, _stream_of(dev))
    if rc:
        _check(rc, "msa_norm_rope_backward")
    return tuple(out_x), tuple(out_w)


def msa_norm_rope_append(xs, weights, inv_freq, seq_len, caches, eps: float = 1e-6, rotate=None,
                         interleaved: bool = False, ws=None, positions=None, axes=None):
    """Norm and rotation of the newest tokens of sequences of lengths seq_len [B] (int32 on the device),
    those with a cache written to their rows of it.

    xs: tensors [B, N, heads, 128] (or [B, heads, 128]: one token), token i at position
    seq_len - N + i.  caches: per tensor a cache [B, S, heads, 128] (one head: also [B, S, 128]) or
    None; a uint8 cache (msa_q4_cache) takes the rows in 4 bits.  positions, axes: as in
    msa_norm_rope_forward, where the tokens' positions are not their rows in the caches (int32 [B, N], or
    [axes, B, N]).  Returns per tensor its cache, or a new tensor of the shape of x: for (q, k, v, qp, kp) with
    caches (None, k_cache, v_cache, None, kp_cache) the arguments of msa_decode and
    msa_window_decode (msa_decode_q4 and msa_window_decode_q4).  Sequences with a length outside N .. S are skipped (msa_device_status of ws
    tells).  Caches may overlap neither each other nor the xs."""
    dev = _device_of(xs)
    x4 = xs
    if xs[0].dim() == 3:
        x4 = [x.unsqueeze(1) if isinstance(x, torch.Tensor) and x.dim() == 3 else x for x in xs]
    shape, parts, fp, pp, axes = _rope_args(x4, weights, rotate, inv_freq, interleaved, eps, positions, dev, axes)
    B = shape.B
    sp = _ask(seq_len, "seq_len", torch.int32, (B,), dev)
    if len(caches) != len(x4):
        raise MSAError("one cache (or None) per tensor")
    capacity = None
    with _Guard(dev):
        outs, rows = [], []
        for i, (at, w, h, f) in enumerate(parts):
            c = caches[i]
            if c is None:
                y = torch.empty(xs[i].shape, dtype=torch.bfloat16, device=dev)
                to = (y.data_ptr(), shape.N * h * 128, h * 128)
                outs.append(y)
            elif isinstance(c, torch.Tensor) and c.dtype is torch.uint8:
                to = (_q4(c, _C_NAMES[i], (B, h), dev), 0, 0)
                if capacity is not None and c.shape[2] * 128 != capacity:
                    raise MSAError(f"caches of different capacities: {capacity}, {c.shape[2] * 128}")
                capacity = c.shape[2] * 128
                f |= ROPE_CACHE_Q4
                outs.append(c)
            else:
                c4 = c.unsqueeze(2) if isinstance(c, torch.Tensor) and c.dim() == 3 else c
                to = _rows(c4, _C_NAMES[i], B, None, h, write=True)
                if c4.device != dev:
                    _on(c4, _C_NAMES[i], dev)
                if capacity is not None and c4.shape[1] != capacity:
                    raise MSAError(f"caches of different capacities: {capacity}, {c4.shape[1]}")
                capacity = c4.shape[1]
                f |= ROPE_CACHE
                outs.append(c)
            rows.append(_PART.pack(*at, *to, 0, 0, 0, w, 0, h, f))
        shape.capacity = 2 ** 31 - 1 if capacity is None else capacity
        wp, wn, ws = _ws(ws, _rope_bytes(len(rows), OP_NORM_ROPE_APPEND), dev)
        if pp is None:
            rc = load_library().msa_norm_rope_append(ctypes.byref(shape), b"".join(rows), len(rows), sp, fp,
                                                     wp, wn, _stream_of(dev))
        else:
            how = None if axes is None else ctypes.byref(axes)
            rc = load_library().msa_norm_rope_axes_append(ctypes.byref(shape), b"".join(rows), len(rows), sp, pp,
                                                          fp, how, wp, wn, _stream_of(dev))
    if rc:
        _check(rc, "msa_norm_rope_append")
    return tuple(outs)


class _NormRopeFunction(torch.autograd.Function):
    """tensors: the weights that are there, then either one packed x (heads given) or the xs."""
    @staticmethod
    def forward(ctx, heads, has_w, inv_freq, positions, eps, rotate, interleaved, axes, *tensors):
        nw = sum(has_w)
        given, xs = list(tensors[:nw]), tensors[nw:]
        weights = [given.pop(0).detach().float().contiguous() if h else None for h in has_w]
        parts = xs[0].split(heads, 2) if heads is not None else xs
        ys = msa_norm_rope_forward(parts, weights, inv_freq, positions, eps, rotate, interleaved, axes)
        ctx.save_for_backward(inv_freq, positions, *xs, *(w for w in weights if w is not None))
        ctx.how = (heads, has_w, eps, rotate, interleaved, axes, len(xs), [t.dtype for t in tensors[:nw]])
        return ys

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, *dys):
        heads, has_w, eps, rotate, interleaved, axes, nx, dtypes = ctx.how
        inv_freq, positions = ctx.saved_tensors[:2]
        xs, saved = ctx.saved_tensors[2:2 + nx], list(ctx.saved_tensors[2 + nx:])
        weights = [saved.pop(0) if h else None for h in has_w]
        if heads is not None:
            dx = torch.empty(xs[0].shape, dtype=xs[0].dtype, device=xs[0].device)
            parts, out = xs[0].split(heads, 2), dx.split(heads, 2)
        else:
            parts, out = xs, None
        dxs, dws = msa_norm_rope_backward(parts, weights, [d.contiguous() for d in dys], inv_freq,
                                          positions, eps, rotate, interleaved, dxs=out, axes=axes)
        grads = tuple(w.to(t) for w, t in zip((w for w in dws if w is not None), dtypes))
        return (None,) * 8 + grads + ((dx,) if heads is not None else dxs)


def _norm_rope_apply(heads, xs, weights, inv_freq, positions, eps, rotate, interleaved, axes):
    n = len(xs) if heads is None else len(heads)
    weights = [None] * n if weights is None else list(weights)
    rotate = None if rotate is None else [bool(r) for r in rotate]
    return _NormRopeFunction.apply(heads, [w is not None for w in weights], inv_freq, positions,
                                   float(eps), rotate, bool(interleaved),
                                   None if axes is None else tuple(axes), *(w for w in weights if w is not None), *xs)


def msa_norm_rope_func(xs, weights, inv_freq, positions=None, eps: float = 1e-6, rotate=None,
                       interleaved: bool = False, axes=None):
    """msa_norm_rope_forward with autograd: gradients of the xs and of the weights (any floating dtype;
    used in fp32)."""
    return _norm_rope_apply(None, tuple(xs), weights, inv_freq, positions, eps, rotate, interleaved, axes)


def msa_norm_rope_packed_func(x, heads, weights, inv_freq, positions=None, eps: float = 1e-6,
                              rotate=None, interleaved: bool = False, axes=None):
    """The same on one packed projection x [B, N, sum(heads), 128]: returns one contiguous tensor per
    entry of heads; the gradient of x is written packed, without a copy."""
    return _norm_rope_apply([int(h) for h in heads], (x,), weights, inv_freq, positions, eps, rotate,
                            interleaved, axes)


# ---------------------------------------------------------------- caches in 4 bits
def msa_q4_cache(B: int, heads: int, capacity: int, device) -> torch.Tensor:
    """An empty cache in 4 bits for B sequences of up to ``capacity`` (a multiple of 128) tokens: uint8
    [B, heads, capacity / 128, 9344], 73 bytes a row (include/msa.h has the format)."""
    B, heads, capacity = int(B), int(heads), int(capacity)
    if not load_library().msa_q4_cache_bytes(B, heads, capacity):
        raise MSAError(load_library().msa_last_error().decode())
    return torch.zeros((B, heads, capacity // 128, Q4_BLOCK_BYTES), dtype=torch.uint8, device=device)


def _q4(t, name, lead, device):
    """t is a cache in 4 bits with these first dimensions; returns its address."""
    if isinstance(t, torch.Tensor) and t.dim() == 4 and t.shape[2] > 0:
        return _ask(t, name, torch.uint8, (*lead, t.shape[2], Q4_BLOCK_BYTES), device)
    _dims(t, name, 4)
    raise MSAError(f"{name} has shape {tuple(t.shape)}, expected a cache of positive capacity")


def msa_q4_read(cache, first: int, count: int):
    """The values that rows first .. first + count - 1 of every sequence stand for: bf16 [B, count, heads, 128]
    (exact: what the decode steps compute with)."""
    B, H = _dims(cache, "cache", 4)[:2]
    dev = cache.device
    if not cache.is_cuda:
        raise MSAError("cache must be a CUDA tensor")
    cp = _q4(cache, "cache", (B, H), dev)
    first, count = int(first), int(count)
    if first < 0 or count < 1 or first + count > cache.shape[2] * 128:
        raise MSAError(f"rows {first} .. {first + count - 1} are not in a cache of {cache.shape[2] * 128}")
    with _Guard(dev):
        out = torch.empty((B, count, H, 128), dtype=torch.bfloat16, device=dev)
        rc = load_library().msa_q4_read(cp, B, H, cache.shape[2] * 128, first, count, out.data_ptr(), _stream_of(dev))
    if rc:
        _check(rc, "msa_q4_read")
    return out


def msa_window_decode_q4(q, k_cache, v_cache, seq_len, window: int, sinks: int, scale: float, ws=None):
    """msa_window_decode over caches in 4 bits (msa_q4_cache, written by msa_norm_rope_append).  Returns
    (o [B, Hq, 128], lse [B, Hq])."""
    B, Hq, D = _dims(q, "q", 3)
    dev = q.device
    if not q.is_cuda:
        raise MSAError("q must be a CUDA tensor")
    _, Hkv, blocks, _ = _dims(k_cache, "k_cache", 4)
    ptrs = (_ask(q, "q", torch.bfloat16, (B, Hq, D), dev), _q4(k_cache, "k_cache", (B, Hkv), dev),
            _ask(v_cache, "v_cache", torch.uint8, k_cache.shape, dev),
            _ask(seq_len, "seq_len", torch.int32, (B,), dev))
    with _Guard(dev):
        shape, need = _window_call(OP_WINDOW_DECODE_Q4, B, blocks * 128, Hq, Hkv, D, _int32(window, "window"),
                                   _int32(sinks, "sinks"), float(scale))
        wp, wn, ws = _ws(ws, need, dev)
        o = torch.empty_like(q)
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
        rc = load_library().msa_window_decode_q4(shape, *ptrs, o.data_ptr(), lse.data_ptr(), wp, wn, _stream_of(dev))
    if rc:
        _check(rc, "msa_window_decode_q4")
    return o, lse


@functools.lru_cache(maxsize=1024)
def _decode_q4_call(*shape):
    return ctypes.byref(Shape(*shape)), msa_workspace_size(Shape(*shape), OP_DECODE_Q4)


def msa_decode_q4(q, qp, k_cache, v_cache, kp_cache, seq_len, top_k: int, scale: float, ws=None):
    """msa_decode with K and V caches in 4 bits (kp_cache [B, S, 1, 128] or [B, S, 128] stays bf16, so the
    selection is the same).  Returns (o [B, Hq, 128], lse [B, Hq], block_idx [B, Hp, top_k])."""
    B, Hq, D = _dims(q, "q", 3)
    Hp = _dims(qp, "qp", 3)[1]
    dev = q.device
    if not q.is_cuda:
        raise MSAError("q must be a CUDA tensor")
    _, Hkv, blocks, _ = _dims(k_cache, "k_cache", 4)
    S = blocks * 128
    if not isinstance(kp_cache, torch.Tensor):
        raise TypeError("kp_cache must be a tensor")
    ptrs = (_ask(q, "q", torch.bfloat16, (B, Hq, D), dev), _ask(qp, "qp", torch.bfloat16, (B, Hp, D), dev),
            _q4(k_cache, "k_cache", (B, Hkv), dev), _ask(v_cache, "v_cache", torch.uint8, k_cache.shape, dev),
            _ask(kp_cache, "kp_cache", torch.bfloat16, (B, S, D) if kp_cache.dim() == 3 else (B, S, 1, D), dev),
            _ask(seq_len, "seq_len", torch.int32, (B,), dev))
    top_k = _int32(top_k, "top_k")
    with _Guard(dev):
        shape, need = _decode_q4_call(B, S, Hq, Hkv, Hp, D, top_k, float(scale))
        wp, wn, ws = _ws(ws, need, dev)
        o = torch.empty_like(q)
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
        idx = torch.empty((B, Hp, top_k), dtype=torch.int32, device=dev)
        rc = load_library().msa_decode_q4(shape, *ptrs, idx.data_ptr(), o.data_ptr(), lse.data_ptr(), wp, wn,
                                          _stream_of(dev))
    if rc:
        _check(rc, "msa_decode_q4")
    return o, lse, idx
