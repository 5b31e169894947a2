"""The 8-bit paged key/value cache: the handle and the torch helpers of the sage_attn_kv_* calls
(include/sage_attn.h says what each computes).

    cache = kv_cache(n_pages, Hkv, D, n_slots, max_pages, page=64, kind="int8")   # empty
    pos = kv_extend(cache, n_new)                 # pages for the new tokens of every slot
    kv_append(cache, k, v, pos, n_new)            # their keys and values, quantized
    o, lse = kv_attention(q, cache)               # their queries
    kv_fork(cache, src), kv_truncate(cache, keep), kv_compact(cache, larger_or_smaller)

Like the other helpers these marshal arguments; everything is computed by the CUDA library on
the current stream of the cache's device.  Errors that only the device can see (too few pages, a number
out of range) are in the cache's status word: get_status(cache.status).
"""
from __future__ import annotations

import ctypes

from . import SAGE_ERR_UNSUPPORTED, SageError, lib, sage_kv_cache

_KINDS = {"int8": 0, "e4m3": 1}


def _arg(t, name, dtype, shape, device):
    """The address of a tensor argument after its checks."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        if t.dtype != dtype or tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: {dtype} of shape {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
        if t.device != device:
            raise ValueError(f"{name}: on {t.device}, the cache is on {device}")
        raise ValueError(f"{name}: not contiguous")
    return t.data_ptr()


class KVCache:
    """One layer's cache over the given tensors (kept alive, never copied).

    k, v: codes [n_pages, Hkv, page, D], int8 or float8_e4m3fn; k_scale, v_scale: fp32 [n_pages, Hkv];
    table: int32 [n_slots, max_pages]; lengths: int32 [n_slots]; refs: int32 [n_pages]; status: int32 [1].
    """

    def __init__(self, k, v, k_scale, v_scale, table, lengths, refs, status):
        import torch
        kinds = {torch.int8: "int8", torch.float8_e4m3fn: "e4m3"}
        if k.dtype not in kinds or k.dim() != 4 or table.dim() != 2:
            raise ValueError("k: int8 or float8_e4m3fn codes [n_pages, Hkv, page, D] and table [n_slots, max_pages] expected")
        if not k.is_cuda:
            raise ValueError("the cache lives on a GPU")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.table, self.lengths, self.refs, self.status = table, lengths, refs, status
        self.kind, self.device = kinds[k.dtype], k.device
        self.n_pages, self.hkv, self.page, self.d = k.shape
        self.n_slots, self.max_pages = table.shape
        dev, f32, i32 = k.device, torch.float32, torch.int32
        scales = (self.n_pages, self.hkv)
        self.c = sage_kv_cache(_arg(k, "k", k.dtype, k.shape, dev), _arg(v, "v", k.dtype, k.shape, dev),
                               _arg(k_scale, "k_scale", f32, scales, dev), _arg(v_scale, "v_scale", f32, scales, dev),
                               _arg(table, "table", i32, table.shape, dev),
                               _arg(lengths, "lengths", i32, (self.n_slots,), dev),
                               _arg(refs, "refs", i32, (self.n_pages,), dev), _arg(status, "status", i32, (1,), dev),
                               self.n_pages, self.hkv, self.page, self.d, self.n_slots, self.max_pages,
                               _KINDS[self.kind])
        self._ref = ctypes.byref(self.c)
        self._slots_shape, self._lib = (self.n_slots,), lib()
        self._i32, self._f32, self._bf16 = i32, f32, torch.bfloat16
        # (the raw handle: torch.cuda.current_stream() alone costs more than a launch)
        self._index, self._device_now, self._stream_of = dev.index, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def kv_cache(n_pages, hkv, d, n_slots, max_pages, page=64, kind="int8", device="cuda") -> KVCache:
    """An empty cache: n_pages pages of `page` tokens for hkv heads, n_slots sequences of at most
    max_pages pages."""
    import torch
    if kind not in _KINDS:
        raise ValueError(f"kind: 'int8' or 'e4m3', got {kind!r}")
    if page not in (16, 32, 64, 128) or d not in (64, 128) or min(n_pages, hkv, n_slots, max_pages) < 1:
        raise SageError("kv_cache", SAGE_ERR_UNSUPPORTED)
    dtype = torch.int8 if kind == "int8" else torch.float8_e4m3fn
    codes = [torch.zeros((n_pages, hkv, page, d), dtype=torch.int8, device=device).view(dtype) for _ in range(2)]
    scales = [torch.zeros((n_pages, hkv), dtype=torch.float32, device=device) for _ in range(2)]
    i32 = {"dtype": torch.int32, "device": device}
    return KVCache(*codes, *scales, torch.zeros((n_slots, max_pages), **i32), torch.zeros(n_slots, **i32),
                   torch.zeros(n_pages, **i32), torch.zeros(1, **i32))


def _call(fn, cache, stream, *args):
    """fn(*args, stream) with the cache's device current and, unless a stream is given, on that
    device's current stream."""
    index = cache._index
    if stream is None and cache._device_now() == index:
        rc = fn(*args, cache._stream_of(index))
    else:
        import torch
        if stream is not None and stream.device != cache.device:
            raise ValueError(f"stream: on {stream.device}, the cache is on {cache.device}")
        with torch.cuda.device(index):
            rc = fn(*args, cache._stream_of(index) if stream is None else stream.cuda_stream)
    if rc:
        raise SageError(fn.__name__, rc)


def _alloc(stream, make, *args, **kw):
    """What `make` allocates for a call on `stream` (None: the current one), out of that stream's own memory: a
    block of the current stream's may have work of that stream before it, which `stream` does not wait for."""
    if stream is None:
        return make(*args, **kw)
    import torch
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _returned(stream, cache, *tensors):
    """Tensors out of the memory of `stream` that the caller gets: once freed they are not given to others
    before what the current stream does with them is done."""
    if stream is not None:
        import torch
        now = torch.cuda.current_stream(cache.device)
        for t in tensors:
            t.record_stream(now)


def _workspace(ws, cache):
    """The checks of a workspace that the caller gives: all of its bytes are written, one behind the other."""
    if ws.device != cache.device:
        raise ValueError(f"ws: on {ws.device}, the cache is on {cache.device}")
    if not ws.is_contiguous():
        raise ValueError("ws: not contiguous")


def _slot_array(t, name, cache):
    return _arg(t, name, cache._i32, cache._slots_shape, cache.device)


def _rows(slots, b, cache):
    """The address of a slots argument (None: batch row b is slot b)."""
    if slots is None:
        if b > cache.n_slots:
            raise ValueError(f"{b} batch rows without slots, the cache has {cache.n_slots}")
        return None
    return _arg(slots, "slots", cache._i32, (b,), cache.device)


def kv_append(cache, k, v, pos, n_new, slots=None, k_shift=None, stream=None):
    """Quantize the first n_new[s] tokens of bf16 k, v [B, Hkv, Nn, D] into the pages of their slots from
    position pos[s] (int32 [n_slots], as kv_extend gives it; a slot that was not extended by so many tokens is
    left alone, SAGE_ERR_INVALID_ARG in the status word).  slots: int32 [B], the slot of each batch row
    (None: row b is slot b); k_shift: fp32 [Hkv, D], subtracted from every key (K-smoothing)."""
    if k.dim() != 4:
        raise ValueError("k, v: [B, Hkv, Nn, D] expected")
    b, _, nn, _ = k.shape
    shape, dev = (b, cache.hkv, nn, cache.d), cache.device
    _call(cache._lib.sage_attn_kv_append, cache, stream, cache._ref, _arg(k, "k", cache._bf16, shape, dev),
          _arg(v, "v", cache._bf16, shape, dev),
          None if k_shift is None else _arg(k_shift, "k_shift", cache._f32, (cache.hkv, cache.d), dev),
          _rows(slots, b, cache), _slot_array(pos, "pos", cache), _slot_array(n_new, "n_new", cache), b, nn)


def alloc_kv_ws(cache, B, H, Nq):
    """Workspace of kv_attention for queries [B, H, Nq, D] on this cache."""
    import torch
    n = lib().sage_attn_kv_ws_bytes(B, H, cache.hkv, cache.d, Nq)
    if n == 0:
        raise SageError("sage_attn_kv_ws_bytes", SAGE_ERR_UNSUPPORTED)
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def kv_attention(q, cache, causal=True, slots=None, q_len=None, sm_scale=None, o=None, lse=None, ws=None, stream=None):
    """Attention of bf16 queries [B, H, Nq, D] over the cache; returns (O bf16, LSE fp32 [B, H, Nq]).
    slots: int32 [B] (None: row b reads slot b); q_len: int32 [B], the queries of each row that count
    (None: Nq; rows behind them are not written); causal: the queries are the newest q_len tokens of
    their sequence, otherwise each sees every key."""
    import torch
    if q.dim() != 4:
        raise ValueError("q: [B, H, Nq, D] expected")
    B, H, Nq, _ = q.shape
    dev = cache.device
    if ws is None:
        ws = _alloc(stream, alloc_kv_ws, cache, B, H, Nq)
    else:
        _workspace(ws, cache)
    if o is None:
        o = _alloc(stream, torch.empty_like, q)
        _returned(stream, cache, o)
    if lse is None:
        lse = _alloc(stream, torch.empty, (B, H, Nq), dtype=torch.float32, device=dev)
        _returned(stream, cache, lse)
    shape = (B, H, Nq, cache.d)
    _call(cache._lib.sage_attn_kv_attention, cache, stream, cache._ref, _arg(q, "q", torch.bfloat16, shape, dev),
          _rows(slots, B, cache), None if q_len is None else _arg(q_len, "q_len", cache._i32, (B,), dev),
          _arg(o, "o", torch.bfloat16, shape, dev), _arg(lse, "lse", torch.float32, (B, H, Nq), dev), ws.data_ptr(),
          ws.nbytes, B, H, Nq, int(causal), 0.0 if sm_scale is None else float(sm_scale))
    return o, lse


def kv_fork(cache, src, stream=None):
    """Slot s with src[s] >= 0 (int32 [n_slots]) takes over the tokens of slot src[s]; pages are shared."""
    _call(cache._lib.sage_attn_kv_fork, cache, stream, cache._ref, _slot_array(src, "src", cache))


def kv_extend(cache, n_new, pos=None, cow=None, stream=None):
    """Room for n_new[s] more tokens in every slot; returns pos (int32 [n_slots]: where they begin, -1
    where the slot could not be served).  cow, if given, receives the shared page that the slot's last
    page was copied from, or -1."""
    import torch
    if pos is None:
        pos = _alloc(stream, torch.empty_like, n_new)
        _returned(stream, cache, pos)
    if cow is None:
        cow = _alloc(stream, torch.empty_like, n_new)
    _call(cache._lib.sage_attn_kv_extend, cache, stream, cache._ref, _slot_array(n_new, "n_new", cache),
          _slot_array(pos, "pos", cache), _slot_array(cow, "cow", cache))
    return pos


def kv_truncate(cache, keep, stream=None):
    """Slot s with keep[s] >= 0 (int32 [n_slots]) keeps its first keep[s] tokens (0: the slot is freed)."""
    _call(cache._lib.sage_attn_kv_truncate, cache, stream, cache._ref, _slot_array(keep, "keep", cache))


def alloc_kv_compact_ws(cache):
    """Workspace of kv_compact from this cache."""
    import torch
    return torch.empty(lib().sage_attn_kv_compact_ws_bytes(cache.n_pages), dtype=torch.uint8, device=cache.device)


def kv_compact(cache, to, ws=None, stream=None):
    """Move the live pages to the front of the pool `to` (a cache of the same geometry, n_pages may
    differ), with tables, lengths and refs."""
    if to.device != cache.device:
        raise ValueError(f"to: on {to.device}, the cache is on {cache.device}")
    if ws is None:
        ws = _alloc(stream, alloc_kv_compact_ws, cache)
    else:
        _workspace(ws, cache)
    _call(cache._lib.sage_attn_kv_compact, cache, stream, cache._ref, to._ref, ws.data_ptr(), ws.nbytes)
