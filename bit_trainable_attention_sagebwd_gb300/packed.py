"""Attention over packed sequences: the torch helpers of the sage_attn_packed_* calls (include/sage_attn.h says what
each computes).

    cu = torch.tensor([0, 700, 700, 1000], dtype=torch.int32, device="cuda")   # three sequences, one of them empty
    o, lse = packed_forward(q, k, v, cu)                                      # q [T, H, D], k, v [T, Hkv, D]
    dq, dk, dv = packed_backward(q, k, v, o, lse, do, cu)

Like the other helpers these marshal arguments; everything is computed by the CUDA library on the current stream of
the tensors' device.  Tensors may be slices of a fused projection or head-major: any strides in multiples of 8
elements with the channels contiguous.  A batch without a token (T = 0) gives empty results, and nothing is launched.
"""
from __future__ import annotations

import ctypes

from . import SAGE_ERR_UNSUPPORTED, SageError, lib

_I64x12, _I64x24 = ctypes.c_longlong * 12, ctypes.c_longlong * 24


def _refuse(x, name, dtype, shape, device, whose="q is"):
    """Why a tensor argument is refused."""
    if x.dtype is not dtype or x.shape != shape:
        raise ValueError(f"{name}: {dtype} of shape {tuple(shape)} expected, got {x.dtype} {tuple(x.shape)}")
    if x.device != device:
        raise ValueError(f"{name}: on {x.device}, {whose} on {device}")
    raise ValueError(f"{name}: not contiguous")


def _rows(x, name, bf16, shape, device):
    """The members of a sage_rows of a tensor argument [T, heads, D], after its checks."""
    token, head, channel = x.stride()
    if x.dtype is not bf16 or x.shape != shape or x.device != device:
        _refuse(x, name, bf16, shape, device)
    if channel != 1:
        raise ValueError(f"{name}: its channels are not contiguous")
    return x.data_ptr(), token, head


def _array(x, name, dtype, shape, device, whose="q is"):
    """The address of a contiguous tensor argument after its checks."""
    if x.dtype is not dtype or x.shape != shape or x.device != device or not x.is_contiguous():
        _refuse(x, name, dtype, shape, device, whose)
    return x.data_ptr()


def _shapes(q, k, cu_seqlens):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q: [T, H, D], k and v: [T, Hkv, D] expected")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens: the S + 1 places where the sequences begin and the last one ends expected")
    if not q.is_cuda:
        raise ValueError("q: on a GPU expected")
    T, H, D = q.shape
    return T, cu_seqlens.shape[0] - 1, H, k.shape[1], D, q.device


def _call(fn, device, stream, *args):
    """fn(*args, stream) with the tensors' device current, on `stream` or that device's current stream."""
    import torch
    if stream is not None and stream.device != device:
        raise ValueError(f"stream: on {stream.device}, q is on {device}")
    if stream is None and torch._C._cuda_getDevice() == device.index:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream)
    if rc:
        raise SageError(fn.__name__, rc)


def _new(stream, device, shape, dtype):
    """A tensor that the caller gets: out of the memory of the stream that the call runs on, and once freed not given
    to others before what the current stream does with it is done."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        x = torch.empty(shape, dtype=dtype, device=device)
    x.record_stream(torch.cuda.current_stream(device))
    return x


def _ws_bytes(T, S, H, Hkv, D, backward):
    """(of no tokens as of one)"""
    n = lib().sage_attn_packed_ws_bytes(T or 1, S, H, Hkv, D, int(backward))
    if n == 0:
        raise SageError("sage_attn_packed_ws_bytes", SAGE_ERR_UNSUPPORTED)
    return n


def alloc_packed_ws(T, S, H, Hkv, D, backward=False, device="cuda", stream=None):
    """Workspace of packed_forward and packed_backward (backward=True) for T tokens in S sequences.  Its status word:
    get_status(ws)."""
    import torch
    n = _ws_bytes(T, S, H, Hkv, D, backward)
    with torch.cuda.stream(stream):
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        ws[:4096].zero_()
    return ws


def _workspace(ws, shape, backward, device, stream):
    if ws is None:
        return alloc_packed_ws(*shape, backward, device, stream)
    if ws.device != device:
        raise ValueError(f"ws: on {ws.device}, q is on {device}")
    if not ws.is_contiguous():
        raise ValueError("ws: not contiguous")
    return ws


def packed_forward(q, k, v, cu_seqlens, causal=True, sm_scale=None, o=None, lse=None, ws=None, stream=None):
    """Attention of every sequence of a packed batch over itself: bf16 q [T, H, D], k and v [T, Hkv, D], int32
    cu_seqlens [S + 1].  Returns (O bf16 [T, H, D], LSE fp32 [H, T]); rows behind the last sequence are left as they
    were.  Entries of cu_seqlens that are out of order or range are reported in the status word of ws."""
    import torch
    T, S, H, Hkv, D, dev = _shapes(q, k, cu_seqlens)
    bf16, qs, kv = torch.bfloat16, (T, H, D), (T, Hkv, D)
    ws = _workspace(ws, (T, S, H, Hkv, D), False, dev, stream)
    if o is None:
        o = _new(stream, dev, qs, bf16)
    if lse is None:
        lse = _new(stream, dev, (H, T), torch.float32)
    rows = _I64x12(*_rows(q, "q", bf16, qs, dev), *_rows(k, "k", bf16, kv, dev), *_rows(v, "v", bf16, kv, dev),
                   *_rows(o, "o", bf16, qs, dev))  # four sage_rows
    at = ctypes.addressof(rows)
    cu_at = _array(cu_seqlens, "cu_seqlens", torch.int32, (S + 1,), dev)
    lse_at = _array(lse, "lse", torch.float32, (H, T), dev)
    if T == 0:
        _ws_bytes(T, S, H, Hkv, D, False)
        return o, lse
    _call(lib().sage_attn_packed_fwd, dev, stream, at, at + 24, at + 48, cu_at, at + 72, lse_at,
          ws.data_ptr(), ws.nbytes, T, S, H, Hkv, D, int(causal), 0.0 if sm_scale is None else float(sm_scale))
    return o, lse


def packed_backward(q, k, v, o, lse, do, cu_seqlens, causal=True, sm_scale=None, dq=None, dk=None, dv=None, ws=None,
                    stream=None):
    """The gradients of packed_forward: from its inputs and results and dO [T, H, D], (dQ, dK, dV) bf16 in the shapes of
    q, k and v.  ws: alloc_packed_ws(.., backward=True)."""
    import torch
    T, S, H, Hkv, D, dev = _shapes(q, k, cu_seqlens)
    bf16, qs, kv = torch.bfloat16, (T, H, D), (T, Hkv, D)
    ws = _workspace(ws, (T, S, H, Hkv, D), True, dev, stream)
    dq = _new(stream, dev, qs, bf16) if dq is None else dq
    dk = _new(stream, dev, kv, bf16) if dk is None else dk
    dv = _new(stream, dev, kv, bf16) if dv is None else dv
    rows = _I64x24(*_rows(q, "q", bf16, qs, dev), *_rows(k, "k", bf16, kv, dev), *_rows(v, "v", bf16, kv, dev),
                   *_rows(o, "o", bf16, qs, dev), *_rows(do, "do", bf16, qs, dev), *_rows(dq, "dq", bf16, qs, dev),
                   *_rows(dk, "dk", bf16, kv, dev), *_rows(dv, "dv", bf16, kv, dev))  # eight sage_rows
    at = ctypes.addressof(rows)
    lse_at = _array(lse, "lse", torch.float32, (H, T), dev)
    cu_at = _array(cu_seqlens, "cu_seqlens", torch.int32, (S + 1,), dev)
    if T == 0:
        _ws_bytes(T, S, H, Hkv, D, True)
        return dq, dk, dv
    _call(lib().sage_attn_packed_bwd, dev, stream, at, at + 24, at + 48, at + 72, lse_at, at + 96, cu_at,
          at + 120, at + 144, at + 168, ws.data_ptr(), ws.nbytes, T, S, H, Hkv, D, int(causal),
          0.0 if sm_scale is None else float(sm_scale))
    return dq, dk, dv
