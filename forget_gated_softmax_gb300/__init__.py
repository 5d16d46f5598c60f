"""Python binding of libfox.so: forget-gated causal softmax attention (FoX) on sm_103a.

Argument marshalling only. Every step of the computation runs in the CUDA
kernels behind the C ABI in include/fox.h; this module turns torch tensors
into pointers, allocates outputs and workspaces when the caller does not pass
them, and raises FoxError on a non-OK status. There is no CPU fallback: if the
library has not been built, every call fails with an error saying so.

Names follow the C ABI: fox_fwd, fox_bwd, fox_fwd_workspace_bytes,
fox_bwd_workspace_bytes, fox_check_error, fox_status_string; fox_cache_append
and fox_decode work on handles made by make_cache and make_batch.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfox.so")

FOX_DTYPE_BF16 = 0
FOX_DTYPE_F32 = 1
FOX_CACHE_ZERO_BYTES = 16384  # of a paged-cache workspace: zero before its first call

STATUS_NAMES = {
    0: "FOX_OK",
    1: "FOX_ERR_INVALID_ARG",
    2: "FOX_ERR_UNSUPPORTED",
    3: "FOX_ERR_WORKSPACE",
    4: "FOX_ERR_CUDA",
    5: "FOX_ERR_TIMEOUT",
    6: "FOX_ERR_DEVICE",
}

# Exported symbols of libfox.so (the entry points include/fox.h declares).
EXPORTS = (
    "fox_fwd",
    "fox_bwd",
    "fox_fwd_workspace_bytes",
    "fox_fwd_min_workspace_bytes",
    "fox_bwd_workspace_bytes",
    "fox_check_error",
    "fox_status_string",
    "fox_version",
    "fox_trace_begin",
    "fox_trace_end",
    "fox_fwd_noalloc",
    "fox_noalloc_check_error",
    "fox_selftest_wait_timeout",
    "fox_noalloc_scratch_bytes",
    "fox_window",
    "fox_window_workspace_bytes",
    "fox_tile_span",
    "fox_gate_proj",
    "fox_fwd_xgate",
    "fox_gate_scan",
    "fox_gate_scan_workspace_bytes",
    "fox_gate_bwd",
    "fox_gate_bwd_workspace_bytes",
    "fox_cache_workspace_bytes",
    "fox_cache_append",
    "fox_cache_append_low",
    "fox_decode",
)


class FoxError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fox_status_string(status)}")


class fox_params(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int),
        ("N", ctypes.c_int),
        ("H", ctypes.c_int),
        ("d", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("bias_from_j", ctypes.c_int),
        ("non_causal", ctypes.c_int),
        ("tile_skip", ctypes.c_int),
        ("gate_ready", ctypes.c_int),
    ]


class fox_cache(ctypes.Structure):
    _fields_ = [
        ("num_pages", ctypes.c_int),
        ("page_size", ctypes.c_int),
        ("H", ctypes.c_int),
        ("Hkv", ctypes.c_int),
        ("d", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("g", ctypes.c_void_p),
        ("gbase", ctypes.c_void_p),
    ]


class fox_batch(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int),
        ("max_new", ctypes.c_int),
        ("table_stride", ctypes.c_int),
        ("prefix_len", ctypes.c_int),
        ("cu_new", ctypes.c_void_p),
        ("lens", ctypes.c_void_p),
        ("table", ctypes.c_void_p),
        ("prefix_table", ctypes.c_void_p),
    ]


class fox_rotary(ctypes.Structure):
    _fields_ = [
        ("cos", ctypes.c_void_p),
        ("sin", ctypes.c_void_p),
        ("max_pos", ctypes.c_int),
        ("dim", ctypes.c_int),
        ("pairs", ctypes.c_int),
        ("q", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64),
        ("q_out", ctypes.c_void_p),
    ]


class fox_trace_record(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char_p), ("ms", ctypes.c_float)]


_lib = None
_call = None  # fox_cache_append_low and fox_decode by way of _foxcall.so (csrc/fox_call.c), or of ctypes without it


def lib() -> ctypes.CDLL:
    """The loaded libfox.so; raises if it has not been built."""
    global _lib, _call
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libfox.so is not built ({LIB_PATH} missing); run "
                "`python -m forget_gated_softmax_gb300.build` (needs nvcc)"
            )
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        pp = ctypes.POINTER(fox_params)
        L.fox_fwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.fox_fwd.restype = i
        L.fox_bwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.fox_bwd.restype = i
        L.fox_fwd_workspace_bytes.argtypes = [pp]
        L.fox_fwd_workspace_bytes.restype = sz
        L.fox_fwd_min_workspace_bytes.argtypes = [pp]
        L.fox_fwd_min_workspace_bytes.restype = sz
        L.fox_bwd_workspace_bytes.argtypes = [pp]
        L.fox_bwd_workspace_bytes.restype = sz
        L.fox_check_error.argtypes = [vp, vp]
        L.fox_check_error.restype = i
        L.fox_status_string.argtypes = [i]
        L.fox_status_string.restype = ctypes.c_char_p
        L.fox_version.argtypes = []
        L.fox_version.restype = i
        L.fox_window_workspace_bytes.argtypes = [pp]
        L.fox_window_workspace_bytes.restype = sz
        L.fox_window.argtypes = [pp, vp, ctypes.c_double, vp, vp, sz, vp]
        L.fox_window.restype = i
        L.fox_gate_proj.argtypes = [pp, i, vp, vp, vp, vp, vp, sz, vp]
        L.fox_gate_proj.restype = i
        L.fox_fwd_xgate.argtypes = [pp, i, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.fox_fwd_xgate.restype = i
        L.fox_tile_span.argtypes = [pp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.fox_tile_span.restype = i
        L.fox_fwd_noalloc.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp]
        L.fox_fwd_noalloc.restype = i
        L.fox_noalloc_scratch_bytes.argtypes = []
        L.fox_noalloc_scratch_bytes.restype = sz
        L.fox_noalloc_check_error.argtypes = [vp]
        L.fox_noalloc_check_error.restype = i
        L.fox_selftest_wait_timeout.argtypes = [ctypes.c_uint, vp, sz, vp]
        L.fox_selftest_wait_timeout.restype = i
        L.fox_gate_scan_workspace_bytes.argtypes = [pp]
        L.fox_gate_scan_workspace_bytes.restype = sz
        L.fox_gate_scan.argtypes = [pp, vp, vp, vp, sz, vp]
        L.fox_gate_scan.restype = i
        L.fox_gate_bwd_workspace_bytes.argtypes = [pp]
        L.fox_gate_bwd_workspace_bytes.restype = sz
        L.fox_gate_bwd.argtypes = [pp, vp, vp, vp, vp, vp, sz, vp]
        L.fox_gate_bwd.restype = i
        pc, pb, i64 = ctypes.POINTER(fox_cache), ctypes.POINTER(fox_batch), ctypes.c_int64
        L.fox_cache_workspace_bytes.argtypes = [pc, pb, i]
        L.fox_cache_workspace_bytes.restype = sz
        L.fox_cache_append.argtypes = [pc, pb, i, vp, i64, vp, i64, vp, i64, ctypes.POINTER(fox_rotary), vp, sz, vp]
        L.fox_cache_append.restype = i
        L.fox_cache_append_low.argtypes = [pc, pb, i, vp, i64, vp, i64, vp, i64, ctypes.POINTER(fox_rotary), vp, vp, sz, vp]
        L.fox_cache_append_low.restype = i
        L.fox_decode.argtypes = [pc, pb, i, vp, i64, ctypes.c_float, i, vp, vp, vp, sz, vp]
        L.fox_decode.restype = i
        try:
            from . import _foxcall
        except ImportError:  # built without Python's headers: libfox.so is all that the calls need
            _call = _CtypesCall
        else:
            _foxcall.bind(*(ctypes.cast(f, vp).value for f in (L.fox_cache_append_low, L.fox_decode)))
            _call = _foxcall
        L.fox_trace_begin.argtypes = []
        L.fox_trace_begin.restype = i
        L.fox_trace_end.argtypes = [ctypes.POINTER(fox_trace_record), i]
        L.fox_trace_end.restype = i
        _lib = L
    return _lib


class _CtypesCall:
    """_foxcall's functions by ctypes, the same numbers in the same order: some microseconds a call longer."""

    @staticmethod
    def append(c, b, rows, k, ks, v, vs, z, zs, ws, nbytes, stream, *more):
        rot = ctypes.byref(fox_rotary(*more[:8])) if len(more) >= 8 else None
        low = more[-1] if len(more) % 8 == 1 else None
        return lib().fox_cache_append_low(ctypes.byref(fox_cache.from_address(c)), ctypes.byref(fox_batch.from_address(b)),
                                          rows, k, ks, v, vs, z, zs, rot, low, ws, nbytes, stream)

    @staticmethod
    def decode(c, b, rows, *more):
        return lib().fox_decode(ctypes.byref(fox_cache.from_address(c)), ctypes.byref(fox_batch.from_address(b)), rows, *more)


def _load_call():
    lib()
    return _call


def fox_status_string(status: int) -> str:
    try:
        return lib().fox_status_string(int(status)).decode()
    except RuntimeError:
        return STATUS_NAMES.get(int(status), f"status {status}")


def make_params(B, N, H, d, dtype=FOX_DTYPE_BF16, scale=0.0, bias_from_j=False, non_causal=False,
                tile_skip=False, gate_ready=False) -> fox_params:
    return fox_params(int(B), int(N), int(H), int(d), int(dtype), float(scale), int(bool(bias_from_j)),
                      int(bool(non_causal)), int(bool(tile_skip)), int(bool(gate_ready)))


def fox_fwd_workspace_bytes(params: fox_params) -> int:
    return int(lib().fox_fwd_workspace_bytes(ctypes.byref(params)))


def fox_fwd_min_workspace_bytes(params: fox_params) -> int:
    return int(lib().fox_fwd_min_workspace_bytes(ctypes.byref(params)))


def fox_bwd_workspace_bytes(params: fox_params) -> int:
    return int(lib().fox_bwd_workspace_bytes(ctypes.byref(params)))


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> Optional[int]:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return FOX_DTYPE_BF16
    if t.dtype == torch.float32:
        return FOX_DTYPE_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def workspace(nbytes: int, device):
    """A 256-byte aligned device workspace of at least nbytes (torch allocation)."""
    torch = _torch()
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def fox_fwd(
    q,
    k,
    v,
    z,
    *,
    scale: float = 0.0,
    bias_from_j: bool = False,
    non_causal: bool = False,
    tile_skip: bool = False,
    o=None,
    lse=None,
    ws=None,
    stream=None,
) -> Tuple[object, object]:
    """Forward: q, k, v [B, N, H, d] (bf16 or fp32), z [B, N, H] fp32 -> (O, LSE).

    O has q's dtype and layout; LSE is fp32 [B, N, H] (natural log). All
    tensors must be contiguous on the current CUDA device.
    """
    torch = _torch()
    B, N, H, d = q.shape
    params = make_params(B, N, H, d, _dtype_code(q), scale, bias_from_j, non_causal, tile_skip)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, N, H), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(fox_fwd_workspace_bytes(params), q.device)
    for t in (q, k, v, z, o, lse):
        if not t.is_contiguous():
            raise ValueError("fox_fwd needs contiguous tensors")
    st = lib().fox_fwd(
        ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
        _stream_handle(stream),
    )
    if st != 0:
        raise FoxError(st, "fox_fwd")
    return o, lse


def fox_bwd(
    q,
    k,
    v,
    z,
    o,
    lse,
    dO,
    *,
    scale: float = 0.0,
    bias_from_j: bool = False,
    non_causal: bool = False,
    tile_skip: bool = False,
    gate_ready: bool = False,
    dq=None,
    dk=None,
    dv=None,
    dz=None,
    ws=None,
    stream=None,
):
    """Backward (bf16): returns (dQ, dK, dV, dz); dz is fp32 [B, N, H]. gate_ready: `ws` holds the
    gate terms of z from a forward on the same workspace (see fox_params.gate_ready)."""
    torch = _torch()
    B, N, H, d = q.shape
    params = make_params(B, N, H, d, _dtype_code(q), scale, bias_from_j, non_causal, tile_skip, gate_ready)
    if gate_ready and ws is None:
        raise ValueError("gate_ready needs the workspace the forward wrote its gate terms into")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    dz = torch.empty((B, N, H), dtype=torch.float32, device=q.device) if dz is None else dz
    if ws is None:
        ws = workspace(fox_bwd_workspace_bytes(params), q.device)
    for t in (q, k, v, z, o, lse, dO, dq, dk, dv, dz):
        if not t.is_contiguous():
            raise ValueError("fox_bwd needs contiguous tensors")
    st = lib().fox_bwd(
        ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
        _ptr(dk), _ptr(dv), _ptr(dz), _ptr(ws), ws.numel(), _stream_handle(stream),
    )
    if st != 0:
        raise FoxError(st, "fox_bwd")
    return dq, dk, dv, dz


def fox_fwd_noalloc(q, k, v, z, *, scale: float = 0.0, bias_from_j: bool = False, o=None, lse=None, stream=None):
    """Forward with the library's fixed device scratch instead of a workspace
    (for callers that cannot allocate device memory; see fox_fwd_noalloc in
    include/fox.h). Output tensors are allocated here only when not passed."""
    torch = _torch()
    B, N, H, d = q.shape
    params = make_params(B, N, H, d, _dtype_code(q), scale, bias_from_j)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, N, H), dtype=torch.float32, device=q.device)
    for t in (q, k, v, z, o, lse):
        if not t.is_contiguous():
            raise ValueError("fox_fwd_noalloc needs contiguous tensors")
    st = lib().fox_fwd_noalloc(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(o), _ptr(lse),
                               _stream_handle(stream))
    if st != 0:
        raise FoxError(st, "fox_fwd_noalloc")
    return o, lse


def fox_window_workspace_bytes(params: fox_params) -> int:
    return int(lib().fox_window_workspace_bytes(ctypes.byref(params)))


def fox_window(z, eps: float, *, window=None, ws=None, stream=None):
    """Epsilon-effective window per query row: z [B, N, H] fp32 -> int32 [B, N, H] (-1: not reached)."""
    torch = _torch()
    B, N, H = z.shape
    params = make_params(B, N, H, 64)
    if window is None:
        window = torch.empty((B, N, H), dtype=torch.int32, device=z.device)
    if ws is None:
        ws = workspace(fox_window_workspace_bytes(params), z.device)
    if not z.is_contiguous() or not window.is_contiguous():
        raise ValueError("fox_window needs contiguous tensors")
    st = lib().fox_window(ctypes.byref(params), _ptr(z), float(eps), _ptr(window), _ptr(ws), ws.numel(),
                          _stream_handle(stream))
    if st != 0:
        raise FoxError(st, "fox_window")
    return window


def fox_gate_scan_workspace_bytes(params: fox_params) -> int:
    return int(lib().fox_gate_scan_workspace_bytes(ctypes.byref(params)))


def fox_gate_scan(z, *, bias_from_j: bool = False, c=None, want_c: bool = True, ws=None, stream=None):
    """The gate step alone: z [B, N, H] fp32 -> the cumulative log gate c [B, N, H] fp32
    (c_t = sum_{l<=t} log sigmoid(z_l)); with want_c=False only the workspace's gate terms
    are formed (what fox_fwd does first) and None is returned."""
    torch = _torch()
    B, N, H = z.shape
    params = make_params(B, N, H, 64, FOX_DTYPE_BF16, 0.0, bias_from_j)
    if want_c and c is None:
        c = torch.empty((B, N, H), dtype=torch.float32, device=z.device)
    if ws is None:
        ws = workspace(fox_gate_scan_workspace_bytes(params), z.device)
    if not z.is_contiguous() or (want_c and not c.is_contiguous()):
        raise ValueError("fox_gate_scan needs contiguous tensors")
    st = lib().fox_gate_scan(ctypes.byref(params), _ptr(z), _ptr(c) if want_c else None, _ptr(ws), ws.numel(),
                             _stream_handle(stream))
    if st != 0:
        raise FoxError(st, "fox_gate_scan")
    return c if want_c else None


def fox_gate_bwd_workspace_bytes(params: fox_params) -> int:
    return int(lib().fox_gate_bwd_workspace_bytes(ctypes.byref(params)))


def fox_gate_bwd(z, R, C, *, bias_from_j: bool = False, dz=None, ws=None, stream=None):
    """Gate gradient from the row / column sums of dS: z [B, N, H] fp32, R and C [B, H, N] fp32
    -> dz [B, N, H] fp32 (suffix sums of R - C, plus C under bias_from_j, times sigmoid(-z))."""
    torch = _torch()
    B, N, H = z.shape
    params = make_params(B, N, H, 64, FOX_DTYPE_BF16, 0.0, bias_from_j)
    if tuple(R.shape) != (B, H, N) or tuple(C.shape) != (B, H, N):
        raise ValueError("fox_gate_bwd: R and C must be [B, H, N]")
    if dz is None:
        dz = torch.empty((B, N, H), dtype=torch.float32, device=z.device)
    if ws is None:
        ws = workspace(fox_gate_bwd_workspace_bytes(params), z.device)
    for t in (z, R, C, dz):
        if not t.is_contiguous():
            raise ValueError("fox_gate_bwd needs contiguous tensors")
    st = lib().fox_gate_bwd(ctypes.byref(params), _ptr(z), _ptr(R), _ptr(C), _ptr(dz), _ptr(ws), ws.numel(),
                            _stream_handle(stream))
    if st != 0:
        raise FoxError(st, "fox_gate_bwd")
    return dz


def fox_gate_proj(x, w_f, b_f, *, bias_from_j: bool = False, z=None, ws=None, stream=None):
    """Gate logits z = x W_f^T + b_f: x [B, N, hidden] bf16, W_f [H, hidden] bf16, b_f [H] fp32
    -> z [B, N, H] fp32 (tensor cores; the gate scan runs in the same kernel into `ws`)."""
    torch = _torch()
    B, N, hidden = x.shape
    H = w_f.shape[0]
    params = make_params(B, N, H, 64, FOX_DTYPE_BF16, 0.0, bias_from_j)
    if z is None:
        z = torch.empty((B, N, H), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(fox_fwd_workspace_bytes(params), x.device)
    for t in (x, w_f, b_f, z):
        if not t.is_contiguous():
            raise ValueError("fox_gate_proj needs contiguous tensors")
    st = lib().fox_gate_proj(ctypes.byref(params), int(hidden), _ptr(x), _ptr(w_f), _ptr(b_f), _ptr(z), _ptr(ws),
                             ws.numel(), _stream_handle(stream))
    if st != 0:
        raise FoxError(st, "fox_gate_proj")
    return z


def fox_fwd_xgate(q, k, v, x, w_f, b_f, *, scale: float = 0.0, bias_from_j: bool = False, tile_skip: bool = False,
                  z=None, o=None, lse=None, ws=None, stream=None):
    """Forward from the gate projection: returns (O, LSE, z) with z = x W_f^T + b_f [B, N, H] fp32."""
    torch = _torch()
    B, N, H, d = q.shape
    hidden = x.shape[-1]
    params = make_params(B, N, H, d, _dtype_code(q), scale, bias_from_j, tile_skip=tile_skip)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, N, H), dtype=torch.float32, device=q.device) if lse is None else lse
    z = torch.empty((B, N, H), dtype=torch.float32, device=q.device) if z is None else z
    if ws is None:
        ws = workspace(fox_fwd_workspace_bytes(params), q.device)
    for t in (q, k, v, x, w_f, b_f, z, o, lse):
        if not t.is_contiguous():
            raise ValueError("fox_fwd_xgate needs contiguous tensors")
    st = lib().fox_fwd_xgate(ctypes.byref(params), int(hidden), _ptr(q), _ptr(k), _ptr(v), _ptr(x), _ptr(w_f),
                             _ptr(b_f), _ptr(z), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(), _stream_handle(stream))
    if st != 0:
        raise FoxError(st, "fox_fwd_xgate")
    return o, lse, z


def fox_tile_span(q, k, z, *, scale: float = 0.0, bias_from_j: bool = False, ws=None, stream=None):
    """Tile spans of the decay-aware tile skip: (jmin, imax), int32 [B*H, ceil(N/128)] each
    (first key tile of every query tile, last query tile of every key tile)."""
    torch = _torch()
    B, N, H, d = q.shape
    params = make_params(B, N, H, d, _dtype_code(q), scale, bias_from_j, tile_skip=True)
    nT = (N + 127) // 128
    jmin = torch.empty((B * H, nT), dtype=torch.int32, device=q.device)
    imax = torch.empty((B * H, nT), dtype=torch.int32, device=q.device)
    if ws is None:
        ws = workspace(fox_fwd_workspace_bytes(params), q.device)
    for t in (q, k, z):
        if not t.is_contiguous():
            raise ValueError("fox_tile_span needs contiguous tensors")
    st = lib().fox_tile_span(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(z), _ptr(jmin), _ptr(imax), _ptr(ws),
                             ws.numel(), _stream_handle(stream))
    if st != 0:
        raise FoxError(st, "fox_tile_span")
    return jmin, imax


# ------------------------------------------------------------------------------- paged cache


class Cache:
    """A paged cache over the caller's tensors (see fox_cache in include/fox.h). Made by make_cache or new_cache."""

    __slots__ = ("k", "v", "g", "gbase", "g_low", "params", "ref", "addr", "device", "index", "dtype", "H", "Hkv", "d", "page_size")


class Batch:
    """One step's sequences over the caller's tensors (see fox_batch in include/fox.h). Made by make_batch.
    The contents of its tensors may change between calls; their storage may not."""

    __slots__ = ("lens", "table", "cu_new", "prefix_table", "params", "ref", "addr", "device", "B")


def make_cache(k, v, g, gbase, g_low=None) -> Cache:
    """A handle on a paged cache: k, v [pages, Hkv, page_size, d] (bf16 or fp32), g [pages, H, page_size] fp32,
    gbase [pages, H, 2] fp32, all contiguous on one CUDA device. g_low, like g, holds what g's rounding leaves of the
    gates' running sums: without it, tokens appended one at a time lose decay behind a strong gate (see fox_cache in
    include/fox.h)."""
    torch = _torch()
    pages, Hkv, S, d = k.shape
    H = g.shape[1]
    if tuple(v.shape) != (pages, Hkv, S, d) or v.dtype != k.dtype:
        raise ValueError("make_cache: v must have k's shape and type")
    if tuple(g.shape) != (pages, H, S) or tuple(gbase.shape) != (pages, H, 2):
        raise ValueError("make_cache: g must be [pages, H, page_size] and gbase [pages, H, 2]")
    if g_low is not None and g_low.shape != g.shape:
        raise ValueError("make_cache: g_low must have g's shape")
    if any(t is not None and t.dtype != torch.float32 for t in (g, gbase, g_low)):
        raise TypeError("make_cache: g, gbase and g_low must be float32")
    for t in (k, v, g, gbase, g_low):
        if t is None:
            continue
        if not t.is_contiguous():
            raise ValueError("make_cache needs contiguous tensors")
        if not t.is_cuda or t.device != k.device:
            raise ValueError("make_cache needs tensors on one CUDA device")
    c = Cache()
    c.g_low = g_low
    c.k, c.v, c.g, c.gbase, c.device, c.index, c.dtype = k, v, g, gbase, k.device, k.device.index, k.dtype
    c.H, c.Hkv, c.d, c.page_size = H, Hkv, d, S
    c.params = fox_cache(pages, S, H, Hkv, d, _dtype_code(k), _ptr(k), _ptr(v), _ptr(g), _ptr(gbase))
    c.ref, c.addr = ctypes.byref(c.params), ctypes.addressof(c.params)
    return c


def new_cache(pages: int, page_size: int, H: int, Hkv: int, d: int, *, dtype=None, device="cuda") -> Cache:
    """make_cache over newly allocated (uninitialised) tensors, g_low among them; dtype defaults to bfloat16."""
    torch = _torch()
    dtype = torch.bfloat16 if dtype is None else dtype
    k, v = (torch.empty((pages, Hkv, page_size, d), dtype=dtype, device=device) for _ in range(2))
    g, g_low = (torch.empty((pages, H, page_size), dtype=torch.float32, device=device) for _ in range(2))
    return make_cache(k, v, g, torch.empty((pages, H, 2), dtype=torch.float32, device=device), g_low)


def make_batch(lens, table, *, cu_new=None, max_new: Optional[int] = None, prefix_table=None,
               prefix_len: int = 0) -> Batch:
    """A handle on a batch: lens [B], table [B, entries], cu_new [B + 1] (None: the same number of rows each),
    prefix_table [ceil(prefix_len / page_size)], int32 on one CUDA device. lens counts every token of a
    sequence, the shared prefix and the new ones among them; 0 is an idle sequence. With cu_new, max_new
    has to say the most new tokens that a sequence may have."""
    torch = _torch()
    B = lens.shape[0]
    if lens.dim() != 1 or table.dim() != 2 or table.shape[0] != B:
        raise ValueError("make_batch: lens must be [B] and table [B, entries]")
    if cu_new is not None and tuple(cu_new.shape) != (B + 1,):
        raise ValueError("make_batch: cu_new must be [B + 1]")
    if cu_new is not None and max_new is None:
        raise ValueError("make_batch: cu_new needs max_new")
    if (prefix_table is None) != (int(prefix_len) == 0):
        raise ValueError("make_batch: prefix_table and prefix_len come together")
    for t in (lens, table, cu_new, prefix_table):
        if t is None:
            continue
        if t.dtype != torch.int32:
            raise TypeError("make_batch: lens, table, cu_new and prefix_table must be int32")
        if not t.is_cuda or t.device != lens.device:
            raise ValueError("make_batch needs tensors on one CUDA device")
        if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError("make_batch needs tensors whose last dimension is contiguous")
    b = Batch()
    b.lens, b.table, b.cu_new, b.prefix_table, b.device, b.B = lens, table, cu_new, prefix_table, lens.device, B
    stride = table.shape[1]
    if not table.is_contiguous():
        raise ValueError("make_batch: table must be contiguous")
    if prefix_table is not None and prefix_table.dim() != 1:
        raise ValueError("make_batch: prefix_table must be one-dimensional")
    b.params = fox_batch(B, 1 if max_new is None else int(max_new), stride, int(prefix_len), _ptr(cu_new), _ptr(lens), _ptr(table),
                         _ptr(prefix_table))
    b.ref, b.addr = ctypes.byref(b.params), ctypes.addressof(b.params)
    return b


def fox_cache_workspace_bytes(cache: Cache, batch: Batch, rows: int) -> int:
    return int(lib().fox_cache_workspace_bytes(cache.ref, batch.ref, int(rows)))


def cache_workspace(cache: Cache, batch: Batch, rows: int):
    """A workspace for fox_cache_append and fox_decode with `rows` rows of this batch, its header zero."""
    n = fox_cache_workspace_bytes(cache, batch, rows)
    if n == 0:
        raise FoxError(1, "cache_workspace")
    ws = workspace(n, cache.device)
    ws[:FOX_CACHE_ZERO_BYTES].zero_()
    return ws


def _cache_call_device(where: str, cache: Cache, batch: Batch) -> int:
    index = cache.index
    if batch.device != cache.device:
        raise ValueError(f"{where}: cache and batch are on different devices")
    if index != _current_device():
        raise ValueError(f"{where}: the cache is not on the current CUDA device")
    if batch.prefix_table is not None and batch.prefix_table.shape[0] * cache.page_size < batch.params.prefix_len:
        raise ValueError(f"{where}: prefix_table has too few pages")
    return index


def _row_stride(where: str, name: str, t, cache: Cache, heads: int, rows: int, index: int) -> int:
    """The stride of t's rows; t is [rows, heads, d] with contiguous rows, in the cache's type, on its device."""
    if t.shape != (rows, heads, cache.d):
        raise ValueError(f"{where}: {name} must be [{rows}, {heads}, {cache.d}], got {tuple(t.shape)}")
    if t.dtype is not cache.dtype:
        raise TypeError(f"{where}: {name} must be {cache.dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{where}: {name} is not on the cache's device")
    s0, s1, s2 = t.stride()
    if (s2 != 1 or (heads > 1 and s1 != cache.d)) and rows:
        raise ValueError(f"{where}: {name} needs contiguous rows")
    return s0


# torch.cuda.current_device() and the current stream's handle, by torch's own short ways where it has them: a
# step of generation is some microseconds of GPU time, of which these would otherwise take three.
def _current_device() -> int:
    global _current_device
    C = _torch()._C
    _current_device = getattr(C, "_cuda_getDevice", None) or _torch().cuda.current_device
    return _current_device()


def _current_stream(index: int) -> int:
    global _current_stream
    torch = _torch()
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _current_stream(index)


def _alloc_on(stream, make):
    """A tensor that the call allocates itself, made in the allocator's order of the stream that uses it."""
    if stream is None:
        return make()
    with _torch().cuda.stream(stream):
        return make()


def fox_cache_append(cache: Cache, batch: Batch, k, v, z, *, q=None, cos=None, sin=None, pairs: bool = False,
                     q_out=None, ws=None, stream=None):
    """Append the batch's new tokens: k, v [rows, Hkv, d] and gate logits z [rows, H] fp32 into the cache's pages.

    cos, sin [positions, r / 2] fp32 rotate the first r channels of k by each token's position on the way
    (channel i with i + r / 2; `pairs`: 2i with 2i + 1), and those of q [rows, H, d] into q_out, which is
    returned (None without q) and must overlap none of the other arguments. Rows may be strided views, as those of
    a joint projection's output. ws: 256 bytes, zero before the first call, or those of cache_workspace; without it what the
    device reports (a page, length or position that does not fit, its token left out) is lost with the call's own."""
    torch = _torch()
    where = "fox_cache_append"
    index = _cache_call_device(where, cache, batch)
    rows = k.shape[0]
    ks = _row_stride(where, "k", k, cache, cache.Hkv, rows, index)
    vs = _row_stride(where, "v", v, cache, cache.Hkv, rows, index)
    f32 = torch.float32
    if z.shape != (rows, cache.H) or z.dtype is not f32 or z.get_device() != index:
        raise ValueError(f"{where}: z must be [{rows}, {cache.H}] float32 on the cache's device")
    zs, z1 = z.stride()
    if z1 != 1 and cache.H > 1 and rows:
        raise ValueError(f"{where}: z needs contiguous rows")
    rot = ()
    if cos is None or sin is None:
        if cos is not None or sin is not None or q is not None or q_out is not None:
            raise ValueError(f"{where}: cos and sin come together, and q only with them")
    else:
        shape = cos.shape
        if len(shape) != 2 or shape != sin.shape or cos.dtype is not f32 or sin.dtype is not f32:
            raise ValueError(f"{where}: cos and sin must be float32 [positions, r / 2]")
        if not (cos.is_contiguous() and sin.is_contiguous() and cos.get_device() == index == sin.get_device()):
            raise ValueError(f"{where}: cos and sin must be contiguous on the cache's device")
        qs = 0
        if q is not None:
            qs = _row_stride(where, "q", q, cache, cache.H, rows, index)
            if q_out is None:
                if stream is None and q.is_contiguous():
                    q_out = torch.empty_like(q)
                else:
                    q_out = _alloc_on(stream, lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device))
            else:
                _row_stride(where, "q_out", q_out, cache, cache.H, rows, index)
                if not q_out.is_contiguous():
                    raise ValueError(f"{where}: q_out must be contiguous")
        elif q_out is not None:
            raise ValueError(f"{where}: q_out without q")
        rot = (cos.data_ptr(), sin.data_ptr(), shape[0], 2 * shape[1], 1 if pairs else 0,
               0 if q is None else q.data_ptr(), qs, 0 if q is None else q_out.data_ptr())
    if cache.g_low is not None:
        rot = (*rot, cache.g_low.data_ptr())
    if ws is None:
        ws = _alloc_on(stream, lambda: torch.zeros(256, dtype=torch.uint8, device=cache.device))
    elif ws.get_device() != index:
        raise ValueError(f"{where}: ws is not on the cache's device")
    st = (_call or _load_call()).append(
        cache.addr, batch.addr, rows, k.data_ptr(), ks, v.data_ptr(), vs, z.data_ptr(), zs, ws.data_ptr(), ws.numel(),
        _current_stream(index) if stream is None else stream.cuda_stream, *rot,
    )
    if st != 0:
        raise FoxError(st, where)
    return q_out


def fox_decode(cache: Cache, batch: Batch, q, *, scale: float = 0.0, bias_from_j: bool = False, o=None, lse=None,
               ws=None, stream=None) -> Tuple[object, object]:
    """Attention of the batch's newest tokens, appended before, over the cache: q [rows, H, d] -> (O [rows, H, d],
    LSE [rows, H] fp32); q, o and lse apart from each other. A long shared prefix is read and multiplied once for all
    sequences (bf16; |v| >= 65536 in it is then reported). Without ws what the device reports is lost.
    Rows of idle sequences get O = 0 and LSE = -inf; rows behind the last sequence are not written."""
    torch = _torch()
    where = "fox_decode"
    index = _cache_call_device(where, cache, batch)
    rows = q.shape[0]
    qs = _row_stride(where, "q", q, cache, cache.H, rows, index)
    if o is None:
        if stream is None and q.is_contiguous():
            o = torch.empty_like(q)
        else:
            o = _alloc_on(stream, lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device))
    else:
        _row_stride(where, "o", o, cache, cache.H, rows, index)
        if not o.is_contiguous():
            raise ValueError(f"{where}: o must be contiguous")
    if lse is None:
        lse = torch.empty((rows, cache.H), dtype=torch.float32, device=cache.device) if stream is None else _alloc_on(
            stream, lambda: torch.empty((rows, cache.H), dtype=torch.float32, device=cache.device))
    elif lse.shape != (rows, cache.H) or lse.dtype is not torch.float32 or lse.get_device() != index or not lse.is_contiguous():
        raise ValueError(f"{where}: lse must be contiguous [{rows}, {cache.H}] float32 on the cache's device")
    if ws is None:
        ws = _alloc_on(stream, lambda: cache_workspace(cache, batch, rows))
    elif ws.get_device() != index:
        raise ValueError(f"{where}: ws is not on the cache's device")
    st = (_call or _load_call()).decode(
        cache.addr, batch.addr, rows, q.data_ptr(), qs, scale, 1 if bias_from_j else 0, o.data_ptr(), lse.data_ptr(),
        ws.data_ptr(), ws.numel(), _current_stream(index) if stream is None else stream.cuda_stream,
    )
    if st != 0:
        raise FoxError(st, where)
    return o, lse


def fox_check_error(ws, stream=None) -> int:
    """Synchronise and read (then clear) the workspace's device error word; returns the status."""
    return int(lib().fox_check_error(_ptr(ws), _stream_handle(stream)))


def fox_noalloc_check_error(stream=None) -> int:
    """fox_check_error for the fixed scratch of fox_fwd_noalloc on the current device."""
    return int(lib().fox_noalloc_check_error(_stream_handle(stream)))


def fox_selftest_wait_timeout(limit_us: int, ws, stream=None) -> None:
    """Enqueue the device error path's self-test (a bounded wait that runs out; see
    fox_selftest_wait_timeout in include/fox.h); read the outcome with fox_check_error(ws)."""
    st = lib().fox_selftest_wait_timeout(int(limit_us), _ptr(ws), ws.numel(), _stream_handle(stream))
    if st != 0:
        raise FoxError(st, "fox_selftest_wait_timeout")


def trace_begin() -> None:
    """Start bracketing every kernel launch of the library with CUDA events (see fox_trace_begin)."""
    st = lib().fox_trace_begin()
    if st != 0:
        raise FoxError(st, "fox_trace_begin")


def trace_end(max_records: int = 1 << 16):
    """Stop tracing; returns [(kernel name, milliseconds)] in launch order."""
    buf = (fox_trace_record * max_records)()
    n = lib().fox_trace_end(buf, max_records)
    if n < 0:
        raise FoxError(4, "fox_trace_end")
    return [(buf[i].kernel.decode(), float(buf[i].ms)) for i in range(min(n, max_records))]
