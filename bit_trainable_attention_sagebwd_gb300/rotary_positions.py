"""Rotary positions: the table of frequencies and the torch helpers of sage_attn_rotary (include/sage_attn.h says what
it computes).

    table = rotary_table(128, scaling="ramp", factor=8.0, context=4096)
    q, k = rotary(table, q, k, cu_seqlens=cu)              # packed [T, H, D]: places in the sequences
    q, k = rotary(table, q, k, start=pos)                  # [B, H, N, D]: pos[b], pos[b] + 1, ... (kv_extend's pos)
    dq, dk = rotary_backward(table, dq, dk, cu_seqlens=cu)

Like the other helpers these marshal arguments; everything but the table is computed by the CUDA library on the
current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import functools
import math

from . import SAGE_ERR_UNSUPPORTED, SageError, lib, sage_rotary
from .packed import _array, _call, _new, _refuse

_I64x8, _I64x16 = ctypes.c_longlong * 8, ctypes.c_longlong * 16
_SCALINGS = ("none", "linear", "base", "ramp")


class Rotary:
    """Frequencies of rotary positions: int64 `turns` [rot / 2] (2^-64 turns a position), the layout of the pairs and the
    factor of the turned channels."""

    def __init__(self, turns, interleaved=False, gain=1.0):
        import torch
        if turns.dtype != torch.int64 or turns.dim() != 1 or not turns.is_contiguous():
            raise ValueError("turns: contiguous int64 [rot / 2] expected")
        if not turns.is_cuda:
            raise ValueError("turns: on a GPU expected")
        self.turns, self.rot, self.interleaved, self.gain = turns, 2 * turns.shape[0], bool(interleaved), float(gain)
        self.device = turns.device
        self.c = sage_rotary(turns.data_ptr(), self.rot, int(self.interleaved), self.gain)
        self._ref = ctypes.byref(self.c)


def rotary_frequencies(rot, base=10000.0, scaling="none", factor=1.0, context=4096, fast=32.0, slow=1.0):
    """(radians a position of each of the rot / 2 pairs as a list, the factor of the turned channels).

    f_c = base^(-2 c / rot), and for contexts `factor` times as long as the one trained at:
      "linear"  f_c / factor (positions interpolated)
      "base"    base times factor^(rot / (rot - 2)): the slowest pair as "linear", the fastest as it was
      "ramp"    pairs that turn more than `fast` times over the trained `context` as they were, fewer than `slow`
                times f_c / factor, between them in proportion to c (the borders on whole pairs, rounded away from
                each other, from pair 0 on); the channels grow by 0.1 ln factor + 1
    """
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling: one of {_SCALINGS}, got {scaling!r}")
    if rot < 4 or rot % 2 or not base > 1 or not factor >= 1:
        raise ValueError("rotary_frequencies: an even rot of 4 at least, base above 1 and factor of 1 at least expected")
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * c / rot) for c in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling != "ramp":
        return f, 1.0
    if not (context > 0 and fast > slow > 0):
        raise ValueError("rotary_frequencies: context above 0 and fast above slow expected")
    first, last = (rot * math.log(context / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow))
    first, last = max(0, math.floor(first)), min(rot - 1, math.ceil(last))
    share = [min(1.0, max(0.0, (c - first) / max(last - first, 1e-3))) for c in range(rot // 2)]
    return [x * (1 - s) + x / factor * s for x, s in zip(f, share)], 0.1 * math.log(factor) + 1.0


@functools.lru_cache(maxsize=8)
def _pi(bits):
    """pi 2^bits, rounded down, by Machin's formula: 16 arctan 1/5 - 4 arctan 1/239."""
    one = 1 << (bits + 32)

    def arctan_of_inverse(n):
        total, power, k = 0, one // n, 0
        while power:
            total += (-1) ** k * (power // (2 * k + 1))
            power //= n * n
            k += 1
        return total

    return (16 * arctan_of_inverse(5) - 4 * arctan_of_inverse(239)) >> 32


def _turns(f):
    """The nearest whole number of 2^-64 turns to f radians, less whole turns: in [-2^63, 2^63)."""
    n, d = abs(f).as_integer_ratio()
    bits = 256 + (n.bit_length() >> 7 << 7)                 # more by 128 than whole turns take
    t = ((n << (64 + bits)) // (d * _pi(bits)) + 1) >> 1    # f / (2 pi) 2^64 and a half, rounded down
    return ((t if f > 0 else -t) + 2 ** 63) % 2 ** 64 - 2 ** 63


def rotary_table(rot, base=10000.0, scaling="none", factor=1.0, context=4096, fast=32.0, slow=1.0, interleaved=False,
                 frequencies=None, gain=None, device="cuda") -> Rotary:
    """The table of rotary_frequencies(rot, ..), or of given `frequencies` (rot / 2 radians a position); `gain` in place
    of the scaling's factor of the turned channels."""
    import torch
    if rot % 16 or not 16 <= rot <= 128:
        raise SageError("rotary_table", SAGE_ERR_UNSUPPORTED)
    if frequencies is None:
        frequencies, of_scaling = rotary_frequencies(rot, base, scaling, factor, context, fast, slow)
    else:
        frequencies, of_scaling = [float(f) for f in frequencies], 1.0
    if len(frequencies) != rot // 2 or not all(math.isfinite(f) for f in frequencies):
        raise ValueError(f"frequencies: {rot // 2} finite numbers expected")
    return Rotary(torch.tensor([_turns(f) for f in frequencies], dtype=torch.int64).to(device), interleaved, of_scaling if gain is None else gain)


def _heads(x, name, bf16, shape, device):
    """The members of a sage_heads of a tensor argument, [T, H, D] or [B, H, N, D], after its checks."""
    stride = x.stride()
    if x.dtype is not bf16 or x.shape != shape or x.device != device:
        _refuse(x, name, bf16, shape, device, "the table is")
    if stride[-1] != 1:
        raise ValueError(f"{name}: its channels are not contiguous")
    if len(stride) == 3:
        return x.data_ptr(), 0, stride[0], stride[1]
    return x.data_ptr(), stride[0], stride[2], stride[1]


def _turn(table, q, k, cu_seqlens, start, positions, q_out, k_out, stream, inverse):
    import torch
    dev = table.device
    if q.dim() not in (3, 4) or (k is not None and k.dim() != q.dim()):
        raise ValueError("q, k: both [T, H, D] or both [B, H, N, D] expected")
    packed = q.dim() == 3
    if packed:
        (N, H, D), B = q.shape, 1
    else:
        B, H, N, D = q.shape
    if cu_seqlens is not None and (not packed or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2):
        raise ValueError("cu_seqlens: [S + 1], with packed [T, H, D] tensors, expected")
    S = 0 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    if table.rot > D:
        raise SageError("rotary", SAGE_ERR_UNSUPPORTED)
    bf16, i32, whose = torch.bfloat16, torch.int32, "the table is"
    if q_out is None:
        q_out = _new(stream, dev, q.shape, bf16)
    heads = _heads(q, "q", bf16, q.shape, dev) + _heads(q_out, "q_out", bf16, q.shape, dev)
    if k is None:
        hkv, heads = 0, _I64x8(*heads)  # two sage_heads
        at = ctypes.addressof(heads)
        keys = keys_out = None
    else:
        hkv = k.shape[1]
        ks = (N, hkv, D) if packed else (B, hkv, N, D)
        if k_out is None:
            k_out = _new(stream, dev, ks, bf16)
        heads = _I64x16(*heads, *_heads(k, "k", bf16, ks, dev), *_heads(k_out, "k_out", bf16, ks, dev))  # four
        at = ctypes.addressof(heads)
        keys, keys_out = at + 64, at + 96
    where = (None if positions is None else _array(positions, "positions", i32, (N,) if packed else (B, N), dev, whose),
             None if start is None else _array(start, "start", i32, (S,) if S else (B,), dev, whose),
             None if cu_seqlens is None else _array(cu_seqlens, "cu_seqlens", i32, (S + 1,), dev, whose))
    if B * N:
        _call(lib().sage_attn_rotary, dev, stream, table._ref, at, at + 32, keys, keys_out, *where, B, N, S, H, hkv, D, inverse)
    elif D not in (64, 128):
        raise SageError("rotary", SAGE_ERR_UNSUPPORTED)
    return q_out if k is None else (q_out, k_out)


def rotary(table, q, k=None, cu_seqlens=None, start=None, positions=None, q_out=None, k_out=None, stream=None):
    """q and k (bf16, both [T, H, D] or both [B, H, N, D]) turned by their positions, in one pass; q_out may be q, k_out k.

    Positions: `positions`, int32 [T] or [B, N]; or start[b] + t (int32 [B]; None: t); or with cu_seqlens (int32 [S + 1],
    packed tensors) a token's place in its sequence + start[s] (int32 [S]); tokens of no sequence are left as they were.
    Returns q_out, with k (q_out, k_out); without a token nothing is launched."""
    return _turn(table, q, k, cu_seqlens, start, positions, q_out, k_out, stream, False)


def rotary_backward(table, dq, dk=None, cu_seqlens=None, start=None, positions=None, q_out=None, k_out=None, stream=None):
    """The gradients of rotary's inputs from those of its outputs: the same call with the angles negated."""
    return _turn(table, dq, dk, cu_seqlens, start, positions, q_out, k_out, stream, True)
