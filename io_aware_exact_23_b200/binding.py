"""ctypes binding of libfa.so: argument marshalling only.

Every function here checks tensor dtypes/shapes/devices, turns torch tensors
into raw device pointers and the current CUDA stream into a handle, and calls
the C entry point of the same name declared in ``include/fa.h`` or ``include/fa_cache.h``.  All
arithmetic happens in the CUDA kernels.  If ``libfa.so`` is missing this module
raises at import: there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa.so")

FA_OK = 0
STATUS_NAMES = {
    0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_MISALIGNED",
    4: "FA_ERR_WORKSPACE", 5: "FA_ERR_NO_DEVICE", 6: "FA_ERR_CUDA", 7: "FA_ERR_DEVICE_TIMEOUT",
    8: "FA_ERR_DEVICE_INTERNAL", 9: "FA_ERR_DEVICE_CACHE",
}


class FaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {lib().fa_status_string(code).decode()} ({code})")


# ``fa_paged_cache`` of include/fa_cache.h, packed into bytes: pointers, strides, then ints.
_PAGED_CACHE = struct.Struct("@4P12q2Pq7i4x")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libfa.so (raises ImportError if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(
                f"{_LIB_PATH} not found: build it with `python -m io_aware_exact_23_b200.build` "
                "(the attention path has no CPU fallback)")
        L = ctypes.CDLL(_LIB_PATH)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_fwd.restype = i
        L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
        L.fa_bwd.restype = i
        L.fa_fwd_residual.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_fwd_residual.restype = i
        L.fa_bwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp,
                                ctypes.POINTER(vp)]
        L.fa_bwd_ex.restype = i
        u64, u32 = ctypes.c_ulonglong, ctypes.c_uint
        L.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_fwd_fp8.restype = i
        L.fa_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, f, u64, u32, vp]
        L.fa_fwd_dropout.restype = i
        L.fa_bwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, f, u64, u32, vp, sz,
                                     vp]
        L.fa_bwd_dropout.restype = i
        L.fa_dropout_mask.argtypes = [i, i, i, f, u64, u32, vp, vp]
        L.fa_dropout_mask.restype = i
        L.fa_bwd_deterministic.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
        L.fa_bwd_deterministic.restype = i
        L.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_bwd_noalloc.restype = i
        L.fa_bwd_workspace_bytes.argtypes = [i, i, i, i]
        L.fa_bwd_workspace_bytes.restype = sz
        L.fa_status_string.argtypes = [i]
        L.fa_status_string.restype = ctypes.c_char_p
        L.fa_device_status.argtypes = [vp]
        L.fa_device_status.restype = i
        L.fa_device_status_info.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
        L.fa_device_status_info.restype = i
        L.fa_selftest_timeout.argtypes = [vp]
        L.fa_selftest_timeout.restype = i
        L.fa_noalloc_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
        L.fa_noalloc_device_status.restype = i
        L.fa_noalloc_selftest_timeout.argtypes = [vp]
        L.fa_noalloc_selftest_timeout.restype = i
        pc = ctypes.c_char_p  # a fa_paged_cache, packed by _paged_cache
        L.fa_cache_append.argtypes = [pc, vp, vp, ctypes.c_char_p, ctypes.c_char_p, i, vp, vp]
        L.fa_cache_append.restype = i
        L.fa_cache_gather.argtypes = [pc, vp, vp, i, i, vp]
        L.fa_cache_gather.restype = i
        L.fa_decode_workspace_bytes.argtypes = [i, i, i, i]
        L.fa_decode_workspace_bytes.restype = sz
        L.fa_decode.argtypes = [pc, vp, vp, vp, i, f, i, vp, sz, vp]
        L.fa_decode.restype = i
        L.fa_version.argtypes = []
        L.fa_version.restype = i
        _lib = L
    return _lib


lib()  # fail at import when the extension is missing


def _stream_handle(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(t: torch.Tensor, name: str, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def fa_fwd(q, k, v, o, lse, scale: float, causal: bool, stream=None, o_lo=None) -> None:
    """O and LSE into the preallocated ``o`` [B,H,N,d] bf16 and ``lse`` [B,H,N] fp32.

    ``o_lo``: optional bf16 tensor shaped like ``o`` that receives O's rounding
    residual (``fa_fwd_residual``), for an exact backward ``D``.
    """
    B, H, N, d = q.shape
    for nm, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    if o_lo is None:
        rc = lib().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                          B, H, N, d, float(scale), int(bool(causal)), _stream_handle(stream))
    else:
        _check(o_lo, "o_lo", torch.bfloat16, (B, H, N, d))
        rc = lib().fa_fwd_residual(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), o_lo.data_ptr(),
                                   lse.data_ptr(), B, H, N, d, float(scale), int(bool(causal)),
                                   _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd")


def fa_fwd_fp8(q8, k8, v8, descale_q, descale_k, descale_v, o, lse, scale: float, causal: bool,
               stream=None) -> None:
    """FP8 forward: ``q8``, ``k8``, ``v8`` are uint8 e4m3 codes [B,H,N,d] (d = 128),
    ``descale_*`` fp32 [B,H] per-head factors (inputs = code * descale); O into the
    bf16 ``o`` [B,H,N,d] and LSE into the fp32 ``lse`` [B,H,N]."""
    B, H, N, d = q8.shape
    for nm, t in (("q8", q8), ("k8", k8), ("v8", v8)):
        _check(t, nm, torch.uint8, (B, H, N, d))
    for nm, t in (("descale_q", descale_q), ("descale_k", descale_k), ("descale_v", descale_v)):
        _check(t, nm, torch.float32, (B, H))
    _check(o, "o", torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    rc = lib().fa_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), descale_q.data_ptr(), descale_k.data_ptr(),
                          descale_v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d, float(scale),
                          int(bool(causal)), _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_fp8")


def fa_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, H, N, d))


def fa_bwd(q, k, v, o, dO, lse, dq, dk, dv, scale: float, causal: bool, workspace, stream=None,
           events=None, o_lo=None) -> None:
    """dQ, dK, dV into preallocated bf16 tensors; ``workspace`` is a uint8 CUDA tensor.

    ``o_lo``: the residual from ``fa_fwd(..., o_lo=...)`` (optional).
    ``events``: optional sequence of four ``torch.cuda.Event(enable_timing=True)``
    recorded around the preprocess, main and dQ-conversion kernels.
    """
    B, H, N, d = q.shape
    for nm, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dO", dO), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    _check(workspace, "workspace", torch.uint8)
    if events is None and o_lo is None:
        rc = lib().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dO.data_ptr(), lse.data_ptr(),
                          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d, float(scale),
                          int(bool(causal)), workspace.data_ptr(), workspace.numel(), _stream_handle(stream))
    else:
        handles = None
        if events is not None:
            if len(events) != 4:
                raise ValueError("events must hold four torch.cuda.Event objects")
            for ev in events:
                if ev.cuda_event == 0:  # torch creates the CUDA event lazily, on first record
                    ev.record()
            handles = (ctypes.c_void_p * 4)(*[ev.cuda_event for ev in events])
        if o_lo is not None:
            _check(o_lo, "o_lo", torch.bfloat16, (B, H, N, d))
        rc = lib().fa_bwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                             None if o_lo is None else o_lo.data_ptr(), dO.data_ptr(), lse.data_ptr(),
                             dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d, float(scale),
                             int(bool(causal)), workspace.data_ptr(), workspace.numel(), _stream_handle(stream),
                             handles)
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd")


def fa_bwd_deterministic(q, k, v, o, dO, lse, dq, dk, dv, scale: float, causal: bool, workspace, stream=None,
                         o_lo=None) -> None:
    """``fa_bwd`` with dQ summed over key tiles in a fixed order: the same bits on
    every call (``fa_bwd_deterministic``); dK and dV are ``fa_bwd``'s."""
    B, H, N, d = q.shape
    for nm, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dO", dO), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    _check(workspace, "workspace", torch.uint8)
    if o_lo is not None:
        _check(o_lo, "o_lo", torch.bfloat16, (B, H, N, d))
    rc = lib().fa_bwd_deterministic(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                    o_lo.data_ptr() if o_lo is not None else None, dO.data_ptr(), lse.data_ptr(),
                                    dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d, float(scale),
                                    int(bool(causal)), workspace.data_ptr(), workspace.numel(),
                                    _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd_deterministic")


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024  # FA_NOALLOC_SCRATCH_BYTES in include/fa.h


def fa_bwd_noalloc(q, k, v, o, dO, lse, dq, dk, dv, scale: float, causal: bool, stream=None) -> None:
    """``fa_bwd`` for callers that cannot allocate device memory: no workspace
    argument; the scratch is a fixed static array inside libfa.so (shapes that
    need more than NOALLOC_SCRATCH_BYTES are refused).  Calls that overlap on
    the GPU share that array and race; the first call on a device does a
    one-time set-up and should come before any stream capture."""
    B, H, N, d = q.shape
    for nm, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dO", dO), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    rc = lib().fa_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dO.data_ptr(),
                              lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d,
                              float(scale), int(bool(causal)), _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd_noalloc")


def fa_noalloc_device_status(stream=None, info: bool = False):
    """Synchronise the stream and return (and clear) fa_bwd_noalloc's own status code."""
    buf = (ctypes.c_int * 4)()
    rc = lib().fa_noalloc_device_status(_stream_handle(stream), buf)
    return (rc, list(buf)) if info else rc


def fa_noalloc_selftest_timeout(stream=None) -> None:
    """The failure-path self-test aimed at fa_bwd_noalloc's status word."""
    rc = lib().fa_noalloc_selftest_timeout(_stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_noalloc_selftest_timeout")


def fa_device_status(stream=None, info: bool = False):
    """Synchronise the stream and return (and clear) the device status code."""
    buf = (ctypes.c_int * 4)()
    rc = lib().fa_device_status_info(_stream_handle(stream), buf)
    return (rc, list(buf)) if info else rc


def fa_selftest_timeout(stream=None) -> None:
    """Launch the failure-path self-test: a wait that gives up after its 1 s limit
    and records FA_ERR_DEVICE_TIMEOUT, which ``fa_device_status`` then returns."""
    rc = lib().fa_selftest_timeout(_stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_selftest_timeout")


class Attention:
    """Allocating convenience wrapper: ``forward`` and ``backward`` on torch tensors."""

    def __init__(self, scale: float, causal: bool):
        self.scale = float(scale)
        self.causal = bool(causal)

    def forward(self, q, k, v, residual: bool = True):
        """Returns (o, lse, o_lo); o_lo is None when ``residual`` is False."""
        B, H, N, d = q.shape
        o = torch.empty_like(q)
        o_lo = torch.empty_like(q) if residual else None
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
        fa_fwd(q, k, v, o, lse, self.scale, self.causal, o_lo=o_lo)
        return o, lse, o_lo

    def backward(self, q, k, v, o, lse, dO, o_lo=None):
        B, H, N, d = q.shape
        ws = torch.empty(fa_bwd_workspace_bytes(B, H, N, d), dtype=torch.uint8, device=q.device)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        fa_bwd(q, k, v, o, dO, lse, dq, dk, dv, self.scale, self.causal, ws, o_lo=o_lo)
        return dq, dk, dv


def fa_fwd_dropout(q, k, v, o, lse, scale: float, causal: bool, rate: float, seed: int, offset: int = 0,
                   stream=None, o_lo=None) -> None:
    """Forward with dropout on the attention probabilities (``fa_fwd_dropout``)."""
    B, H, N, d = q.shape
    for nm, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    if o_lo is not None:
        _check(o_lo, "o_lo", torch.bfloat16, (B, H, N, d))
    rc = lib().fa_fwd_dropout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              o_lo.data_ptr() if o_lo is not None else None, lse.data_ptr(), B, H, N, d,
                              float(scale), int(bool(causal)), float(rate), int(seed) & (2**64 - 1),
                              int(offset) & 0xFFFFFFFF, _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_dropout")


def fa_bwd_dropout(q, k, v, o, dO, lse, dq, dk, dv, scale: float, causal: bool, rate: float, seed: int,
                   workspace, offset: int = 0, stream=None, o_lo=None) -> None:
    """Backward of ``fa_fwd_dropout`` (the mask is regenerated from rate, seed and offset)."""
    B, H, N, d = q.shape
    for nm, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dO", dO), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check(t, nm, torch.bfloat16, (B, H, N, d))
    _check(lse, "lse", torch.float32, (B, H, N))
    _check(workspace, "workspace", torch.uint8)
    if o_lo is not None:
        _check(o_lo, "o_lo", torch.bfloat16, (B, H, N, d))
    rc = lib().fa_bwd_dropout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              o_lo.data_ptr() if o_lo is not None else None, dO.data_ptr(), lse.data_ptr(),
                              dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d, float(scale),
                              int(bool(causal)), float(rate), int(seed) & (2**64 - 1), int(offset) & 0xFFFFFFFF,
                              workspace.data_ptr(), workspace.numel(), _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd_dropout")


def fa_dropout_mask(B: int, H: int, N: int, rate: float, seed: int, offset: int, mask, stream=None) -> None:
    """keep[b, h, i, j] in {0, 1} into the uint8 CUDA tensor ``mask`` [B,H,N,N]."""
    _check(mask, "mask", torch.uint8, (B, H, N, N))
    rc = lib().fa_dropout_mask(B, H, N, float(rate), int(seed) & (2**64 - 1), int(offset) & 0xFFFFFFFF,
                               mask.data_ptr(), _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_dropout_mask")


# ------------------------------------------------------------ key/value cache
# A decode step calls these once a layer and little else happens on the host, so the checks
# are written for the case that they hold: each tensor is looked at in line, and _check_on
# says what is wrong with one that does not pass (or accepts a subclass of Tensor).
CACHE_BF16, CACHE_E4M3 = 0, 1
_STRIDES2 = struct.Struct("@2q")
_Tensor, _BF16, _U8, _I32, _F32 = torch.Tensor, torch.bfloat16, torch.uint8, torch.int32, torch.float32
_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _check_on(t, name: str, dtype, shape, device: int):
    """Type, device and shape of a tensor whose strides the caller deals with."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _paged_cache(k, v, block_table, seq_lens, k_scale, v_scale):
    """The packed C description of a cache held in torch tensors (any strides with adjacent
    row elements), and (device, B, H, d)."""
    if not isinstance(k, _Tensor) or not isinstance(block_table, _Tensor):
        raise TypeError("k_cache and block_table must be torch.Tensor")
    dt, dev, shape, table = k.dtype, k.get_device(), k.shape, block_table.shape
    if dt is not _BF16 and dt is not _U8:
        raise TypeError(f"k_cache must be torch.bfloat16 or torch.uint8 (e4m3 codes), got {dt}")
    if dev < 0:
        raise ValueError("k_cache must be a CUDA tensor")
    if len(shape) != 4 or len(table) != 2:
        raise ValueError("k_cache is [pages, H, page_size, d] and block_table [B, max_pages]")
    P, H, page, d = shape
    B, per = table
    if not (type(v) is _Tensor and v.dtype is dt and v.get_device() == dev and v.shape == shape):
        _check_on(v, "v_cache", dt, shape, dev)
    if not (block_table.dtype is _I32 and block_table.get_device() == dev):
        _check_on(block_table, "block_table", _I32, table, dev)
    if not (type(seq_lens) is _Tensor and seq_lens.dtype is _I32 and seq_lens.get_device() == dev and
            seq_lens.shape == (B,)):
        _check_on(seq_lens, "seq_lens", _I32, (B,), dev)
    k0, k1, k2, k3 = k.stride()
    v0, v1, v2, v3 = v.stride()
    b0, b1 = block_table.stride()
    if (d > 1 and (k3 != 1 or v3 != 1)) or (per > 1 and b1 != 1) or (B > 1 and seq_lens.stride(0) != 1):
        raise ValueError("the last dimension of k_cache, v_cache, block_table and seq_lens must be contiguous")
    if dt is _BF16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("k_scale and v_scale belong to a cache of e4m3 codes (torch.uint8)")
        return _PAGED_CACHE.pack(k.data_ptr(), v.data_ptr(), 0, 0, k0, k1, k2, v0, v1, v2, 0, 0, 0, 0, 0, 0,
                                 block_table.data_ptr(), seq_lens.data_ptr(), b0, CACHE_BF16, P, H, page, d, B,
                                 per), dev, B, H, d
    rows = (P, H, page)
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if not (type(t) is _Tensor and t.dtype is _F32 and t.get_device() == dev and t.shape == rows):
            _check_on(t, name, _F32, rows, dev)
    return _PAGED_CACHE.pack(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k0, k1, k2, v0, v1, v2,
                             *k_scale.stride(), *v_scale.stride(), block_table.data_ptr(), seq_lens.data_ptr(), b0,
                             CACHE_E4M3, P, H, page, d, B, per), dev, B, H, d


def _call_on(device: int, where: str, stream, fn, *args) -> None:
    """Call a C entry point with ``device`` current, on ``stream`` (its current stream by default)."""
    if stream is None:
        handle = _raw_stream(device)
    elif stream.device.index != device:
        raise ValueError(f"{where}: the stream is on {stream.device}, the tensors on cuda:{device}")
    else:
        handle = stream.cuda_stream
    if _current_device() == device:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    if rc != FA_OK:
        raise FaError(rc, where)


def fa_cache_append(k_new, v_new, k_cache, v_cache, block_table, seq_lens, cu_new=None, k_scale=None, v_scale=None,
                    stream=None) -> None:
    """Write new tokens' keys and values into a paged cache.

    ``k_new``, ``v_new``: bf16 [T, H, d] (adjacent row elements; other strides free);
    ``k_cache``, ``v_cache``: [pages, H, page_size, d] bf16, or uint8 e4m3 codes with
    fp32 factors ``k_scale``, ``v_scale`` [pages, H, page_size] (permuted views of
    other layouts welcome); ``block_table`` [B, max_pages] and ``seq_lens`` [B] int32,
    the lengths after the write.  ``cu_new`` None: one token per sequence (T = B);
    else int32 [B + 1], tokens ``cu_new[b]:cu_new[b+1]`` end sequence b.
    """
    c, dev, B, H, d = _paged_cache(k_cache, v_cache, block_table, seq_lens, k_scale, v_scale)
    if not isinstance(k_new, _Tensor) or k_new.dim() != 3:
        raise ValueError("k_new must be a [T, H, d] tensor")
    T = k_new.shape[0]
    rows = (T, H, d)
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if not (type(t) is _Tensor and t.dtype is _BF16 and t.get_device() == dev and t.shape == rows):
            _check_on(t, name, _BF16, rows, dev)
    k0, k1, k2 = k_new.stride()
    v0, v1, v2 = v_new.stride()
    if T and (k2 != 1 or v2 != 1):
        raise ValueError("the last dimension of k_new and v_new must be contiguous")
    cu = None
    if cu_new is not None:
        _check_on(cu_new, "cu_new", _I32, (B + 1,), dev)
        if not cu_new.is_contiguous():
            raise ValueError("cu_new must be contiguous")
        cu = cu_new.data_ptr()
    elif T != B:
        raise ValueError(f"k_new has {T} tokens for {B} sequences: pass cu_new")
    _call_on(dev, "fa_cache_append", stream, _lib.fa_cache_append, c, k_new.data_ptr(), v_new.data_ptr(),
             _STRIDES2.pack(k0, k1), _STRIDES2.pack(v0, v1), T, cu)


def fa_cache_gather(k_cache, v_cache, block_table, seq_lens, k_out, v_out, k_scale=None, v_scale=None,
                    stream=None) -> None:
    """Read sequences back from a paged cache into contiguous bf16 [B, H * rep, N, d] tensors.

    The first N positions of each sequence, zeros behind its end, each cache head
    repeated ``rep`` times (from the outputs' shape): the K and V that ``fa_fwd``
    takes.  ``k_out`` or ``v_out`` may be None.  The cache is as in ``fa_cache_append``.
    """
    c, dev, B, H, d = _paged_cache(k_cache, v_cache, block_table, seq_lens, k_scale, v_scale)
    out = k_out if k_out is not None else v_out
    if not isinstance(out, _Tensor) or out.dim() != 4 or out.shape[1] % H != 0:
        raise ValueError(f"k_out and v_out are [B, {H} * rep, N, d] tensors, and one of them is needed")
    _, heads, N, _ = out.shape
    shape = (B, heads, N, d)
    ptrs = []
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is None:
            ptrs.append(None)
            continue
        if not (type(t) is _Tensor and t.dtype is _BF16 and t.get_device() == dev and t.shape == shape):
            _check_on(t, name, _BF16, shape, dev)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        ptrs.append(t.data_ptr())
    _call_on(dev, "fa_cache_gather", stream, _lib.fa_cache_gather, c, ptrs[0], ptrs[1], heads // H, N)


def fa_decode_workspace_bytes(B: int, Hq: int, H: int, d: int) -> int:
    return int(lib().fa_decode_workspace_bytes(B, Hq, H, d))


def fa_decode(q, k_cache, v_cache, block_table, seq_lens, o, lse, scale: float, workspace, k_scale=None, v_scale=None,
              window: int = 0, stream=None) -> None:
    """Attention of one new token per sequence over a paged cache.

    ``q``, ``o``: bf16 [B, Hq, d], Hq a multiple of the cache's heads; ``lse``: fp32
    [B, Hq] or None; ``workspace``: uint8, ``fa_decode_workspace_bytes`` long;
    ``window``: how many of a sequence's last positions are seen (0: all).  ``o`` may be
    ``q`` itself.  The cache is as in ``fa_cache_append``, the new token's key and value
    already in it.
    """
    c, dev, B, _, d = _paged_cache(k_cache, v_cache, block_table, seq_lens, k_scale, v_scale)
    if not isinstance(q, _Tensor) or q.dim() != 3:
        raise ValueError("q must be a [B, Hq, d] tensor")
    Hq = q.shape[1]
    shape = (B, Hq, d)
    for name, t in (("q", q), ("o", o)):
        if not (type(t) is _Tensor and t.dtype is _BF16 and t.get_device() == dev and t.shape == shape):
            _check_on(t, name, _BF16, shape, dev)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    lse_ptr = None
    if lse is not None:
        if not (type(lse) is _Tensor and lse.dtype is _F32 and lse.get_device() == dev and lse.shape == (B, Hq)):
            _check_on(lse, "lse", _F32, (B, Hq), dev)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
        lse_ptr = lse.data_ptr()
    if not (type(workspace) is _Tensor and workspace.dtype is _U8 and workspace.get_device() == dev):
        _check_on(workspace, "workspace", _U8, None, dev)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if not 0 <= window <= 0x7FFFFFFF:  # ctypes would keep the low 32 bits: more than any length, or refused
        window = 0 if window > 0 else -1
    _call_on(dev, "fa_decode", stream, _lib.fa_decode, c, q.data_ptr(), o.data_ptr(), lse_ptr, Hq, scale, window,
             workspace.data_ptr(), workspace.numel())


_AS_IT_IS = contextlib.nullcontext()


class KVCache:
    """Allocating convenience wrapper of a paged cache: its tensors and the calls on them.

    The caller owns the pages' allocation: ``block_table`` [B, max_pages] and ``seq_lens``
    [B] (int32, the cache's device) go with every call.
    """

    def __init__(self, num_pages: int, H: int, page_size: int, d: int, e4m3: bool = False, device="cuda"):
        shape = (num_pages, H, page_size, d)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8 if e4m3 else torch.bfloat16, device=device)
                          for _ in range(2))
        self.k_scale = self.v_scale = None
        if e4m3:
            self.k_scale, self.v_scale = (torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2))

    def append(self, k_new, v_new, block_table, seq_lens, cu_new=None, stream=None) -> None:
        fa_cache_append(k_new, v_new, self.k, self.v, block_table, seq_lens, cu_new, self.k_scale, self.v_scale, stream)

    def decode(self, q, block_table, seq_lens, scale: float, window: int = 0, stream=None):
        """Returns (o, lse), as on ``stream`` (its memory is that stream's)."""
        B, Hq, d = q.shape
        with torch.cuda.stream(stream) if stream is not None else _AS_IT_IS:
            o = torch.empty_like(q)
            lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
            ws = torch.empty(fa_decode_workspace_bytes(B, Hq, self.k.shape[1], d), dtype=torch.uint8, device=q.device)
            fa_decode(q, self.k, self.v, block_table, seq_lens, o, lse, scale, ws, self.k_scale, self.v_scale, window, stream)
        return o, lse

    def gather(self, block_table, seq_lens, N: int, rep: int = 1, stream=None):
        """Returns (k, v), each [B, H * rep, N, d] bf16, as on ``stream``."""
        _, H, _, d = self.k.shape
        with torch.cuda.stream(stream) if stream is not None else _AS_IT_IS:
            k, v = (torch.empty((block_table.shape[0], H * rep, N, d), dtype=torch.bfloat16, device=self.k.device)
                    for _ in range(2))
            fa_cache_gather(self.k, self.v, block_table, seq_lens, k, v, self.k_scale, self.v_scale, stream)
        return k, v
