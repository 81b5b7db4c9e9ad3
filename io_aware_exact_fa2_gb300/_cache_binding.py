"""ctypes binding to libfa2_cache_gb300.so (declared in include/fa2_cache.h): the paged
8-bit key/value cache and attention over it.

Argument marshalling only, as in ``_binding``: shape, dtype and device checks, raw
pointers, the current CUDA stream; there is no fallback.  Importing this module raises
ImportError if the library has not been built.

A step's kernels take microseconds, so the checks are written for speed: each attribute of
a tensor is read once, and structures are packed rather than built field by field (a call
takes 8 to 10 us of host time, 3 to 5 of them in the library; plainly written it took 22).
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from ._binding import Fa2Error, _stream_handle
from .build import CACHE_LIB_PATH

_vp, _i = ctypes.c_void_p, ctypes.c_int


# struct fa2_cache: pointers k, v, k_scale, v_scale, page_table; (page, head, slot) strides of
# keys and of values; num_pages, H, page_size, D, B, max_pages
_pack_cache = struct.Struct("=5Q6q6i").pack
_pack_strides = struct.Struct("=3q").pack


def load_cache_library() -> ctypes.CDLL:
    if not os.path.exists(CACHE_LIB_PATH):
        raise ImportError(
            f"CUDA library {CACHE_LIB_PATH} is missing: build it with "
            "`python -m io_aware_exact_fa2_gb300.build` (there is no CPU fallback)")
    lib = ctypes.CDLL(CACHE_LIB_PATH)
    sz = ctypes.c_size_t
    for name in ("fa2_cache_write", "fa2_cache_read"):
        f = getattr(lib, name)
        f.restype = _i
        f.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp]
    lib.fa2_cache_attn.restype = _i
    lib.fa2_cache_attn.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, ctypes.c_float, _vp, sz, _vp]
    lib.fa2_cache_attn_workspace_size.restype = _i
    lib.fa2_cache_attn_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i, ctypes.POINTER(sz)]
    lib.fa2_cache_get_device_error.restype = _i
    lib.fa2_cache_get_device_error.argtypes = [_vp, ctypes.POINTER(_i)]
    return lib


_lib = load_cache_library()
_CODES, _BF16, _I32 = torch.float8_e4m3fn, torch.bfloat16, torch.int32
_SCALES = (torch.float8_e8m0fnu, torch.uint8)
_MAX_ROWS = 1 << 30   # of a sequence (the library's limit; checked here, too, for it takes an int)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def cache_library_path() -> str:
    return CACHE_LIB_PATH


def _stream(stream, dev):
    return _raw_stream(dev) if stream is None else _stream_handle(stream, dev)


def _strides(t, shape, unit):
    """The first three strides of a 4-D view whose rows are contiguous.  A dimension of
    size one is never stepped over, so its stride is whatever the library accepts."""
    a, b, c, d = t.stride()
    if d != 1:
        raise ValueError("the last dimension must be contiguous")
    if 1 in shape:
        m, n, o, _ = shape
        if m == 1:
            a = unit
        if n == 1:
            b = unit
        if o == 1:
            c = unit
    return a, b, c


def _cache(k_cache, v_cache, k_scale, v_scale, page_table):
    """struct fa2_cache (its bytes), the device, and B, H, D."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be (pages, H, page_size, D) views of one shape")
    if k_cache.dtype is not _CODES or v_cache.dtype is not _CODES:
        raise TypeError("k_cache and v_cache must be float8_e4m3fn")
    if k_scale.dtype not in _SCALES or v_scale.dtype not in _SCALES:
        raise TypeError("k_scale and v_scale must be float8_e8m0fnu (or its bytes, uint8)")
    dev = k_cache.get_device()
    if dev < 0 or not dev == v_cache.get_device() == k_scale.get_device() == v_scale.get_device() == page_table.get_device():
        raise ValueError("the cache, its scales and page_table must be on one CUDA device")
    N, H, P, D = shape
    if k_scale.shape != (N, H) or v_scale.shape != (N, H) or not k_scale.is_contiguous() or not v_scale.is_contiguous():
        raise ValueError("k_scale and v_scale must be contiguous (pages, H)")
    table = page_table.shape
    if len(table) != 2 or page_table.dtype is not _I32 or not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 (B, max_pages) tensor")
    B, M = table
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), page_table.data_ptr(),
                       *_strides(k_cache, shape, 16), *_strides(v_cache, shape, 16), N, H, P, D, B, M), dev, B, H, D


def _lengths(name, t, B, dev):
    if t.dtype is not _I32 or t.shape != (B,) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 ({B},) tensor on the cache's device")
    return t.data_ptr()


def _rows(name, t, shape, dev):
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must have shape {tuple(shape)} on the cache's device, got {tuple(t.shape)}")
    return _pack_strides(*_strides(t, shape, 8))


def _move(call, where, k_cache, v_cache, k_scale, v_scale, page_table, k, v, starts, counts, stream):
    c, dev, B, H, D = _cache(k_cache, v_cache, k_scale, v_scale, page_table)
    if k.ndim != 4:
        raise ValueError("k and v must be 4-D (B, H, L, D) views")
    L = k.shape[2]
    if L > _MAX_ROWS:
        raise ValueError("k and v must have at most 2^30 rows a sequence")
    shape = (B, H, L, D)
    ks, vs = _rows("k", k, shape, dev), _rows("v", v, shape, dev)
    starts = _lengths("starts", starts, B, dev)
    if counts is not None:
        counts = _lengths("counts", counts, B, dev)
    if L == 0:   # (an empty tensor has no address)
        return
    st = call(c, k.data_ptr(), v.data_ptr(), ks, vs, starts, counts, L, _stream(stream, dev))
    if st != 0:
        raise Fa2Error(st, where)


def fa2_cache_write(k, v, k_cache, v_cache, k_scale, v_scale, page_table, starts, counts=None, stream=None) -> None:
    """Quantise new keys and values into the cache (fa2_cache_write).

    k, v: (B, H, L, D) bfloat16 views with contiguous rows.  k_cache, v_cache:
    (pages, H, page_size, D) float8_e4m3fn views with contiguous rows (so slot-major
    storage is passed permuted).  k_scale, v_scale: (pages, H) float8_e8m0fnu.
    page_table: (B, max_pages) int32.  Row i < counts[b] (default L) of sequence b goes to
    position starts[b] + i; both are (B,) int32.
    """
    _move(_lib.fa2_cache_write, "fa2_cache_write", k_cache, v_cache, k_scale, v_scale, page_table, k, v, starts, counts, stream)


def fa2_cache_read(k_cache, v_cache, k_scale, v_scale, page_table, k, v, starts, counts=None, stream=None) -> None:
    """Read keys and values out of the cache (fa2_cache_read): row i < counts[b] (default L)
    of the (B, H, L, D) bfloat16 views k and v gets position starts[b] + i of sequence b."""
    _move(_lib.fa2_cache_read, "fa2_cache_read", k_cache, v_cache, k_scale, v_scale, page_table, k, v, starts, counts, stream)


def fa2_cache_attn(q, k_cache, v_cache, k_scale, v_scale, page_table, kv_lens, o, lse, causal: bool = True,
                   q_lens=None, window: int | None = None, scale: float | None = None, workspace=None,
                   stream=None) -> None:
    """Attention of the newest tokens over the cache (fa2_cache_attn): writes o and lse.

    q, o: (B, Hq, Lq, D) bfloat16 views with contiguous rows, Hq a multiple of the cache's
    H; lse: contiguous (B, Hq, Lq) float32.  kv_lens: (B,) int32, positions each sequence
    holds, its query tokens among them; q_lens: (B,) int32 rows of each (default Lq), the
    last ones held.  With `workspace` (from fa2_cache_attn_workspace) the keys of one
    sequence are shared out among SMs.
    """
    c, dev, B, H, D = _cache(k_cache, v_cache, k_scale, v_scale, page_table)
    if q.ndim != 4:
        raise ValueError("q and o must be 4-D (B, Hq, Lq, D) views")
    Hq, Lq = q.shape[1:3]
    if Lq > _MAX_ROWS:
        raise ValueError("q and o must have at most 2^30 rows a sequence")
    shape = (B, Hq, Lq, D)
    qs, os_ = _rows("q", q, shape, dev), _rows("o", o, shape, dev)
    if lse.dtype is not torch.float32 or lse.shape != (B, Hq, Lq) or lse.get_device() != dev or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, Hq, Lq) tensor on the cache's device")
    kv_lens = _lengths("kv_lens", kv_lens, B, dev)
    if q_lens is not None:
        q_lens = _lengths("q_lens", q_lens, B, dev)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous and on the cache's device")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.nbytes
    if Lq == 0:   # (an empty tensor has no address)
        return
    # (a window past the longest sequence hides nothing; -2 is refused)
    st = _lib.fa2_cache_attn(c, q.data_ptr(), o.data_ptr(), lse.data_ptr(), qs, os_, kv_lens, q_lens, Hq, Lq, bool(causal),
                             -1 if window is None else max(-2, min(int(window), _MAX_ROWS)), D ** -0.5 if scale is None else scale, ws_ptr, ws_bytes,
                             _stream(stream, dev))
    if st != 0:
        raise Fa2Error(st, "fa2_cache_attn")


def fa2_cache_attn_workspace_size(B: int, Hq: int, H: int, Lq: int, D: int, device: int = 0) -> int:
    """Bytes of workspace fa2_cache_attn can use on `device`, whatever the lengths."""
    n = ctypes.c_size_t(0)
    st = _lib.fa2_cache_attn_workspace_size(B, Hq, H, Lq, D, int(device), ctypes.byref(n))
    if st != 0:
        raise Fa2Error(st, "fa2_cache_attn_workspace_size")
    return int(n.value)


def fa2_cache_attn_workspace(q, k_cache):
    """A zero-filled uint8 CUDA tensor sized for fa2_cache_attn on q's problem.  Keep it
    between calls; calls that may overlap on the GPU need one each.  It is filled on the
    current stream: a first call on another one has to wait for that."""
    B, Hq, Lq, D = q.shape
    n = fa2_cache_attn_workspace_size(B, Hq, k_cache.shape[1], Lq, D, q.device.index or 0)
    return torch.zeros(n, dtype=torch.uint8, device=q.device)


def fa2_cache_get_device_error(stream=None) -> tuple[int, int]:
    """Synchronise, then read and clear the cache kernels' error word: (status, raw code)."""
    detail = ctypes.c_int(0)
    st = _lib.fa2_cache_get_device_error(_stream_handle(stream, torch.cuda.current_device()), ctypes.byref(detail))
    return st, detail.value
