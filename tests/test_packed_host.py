"""Packed attention and rotary positions without a GPU: the entry points refuse bad arguments before anything is launched,
the workspaces have their sizes, the helpers check their tensors, and the frequencies are what they are said to be."""
import ctypes
import math

import pytest
import torch

import bit_trainable_attention_sagebwd_gb300 as sa


@pytest.fixture(scope="module")
def lib():
    from bit_trainable_attention_sagebwd_gb300 import build
    build.build()
    return sa.lib()


FAKE = 0x10000  # aligned, never dereferenced: the checks fail first
NULL_ROWS = NULL_HEADS = None


def rows(p=FAKE, token=512, head=128):
    return sa.sage_rows(p, token, head)


SHAPE = dict(T=300, S=3, H=4, Hkv=2, D=128)


def forward(**o):
    s = SHAPE | {n: o[n] for n in SHAPE if n in o}
    t = {n: o.get(n, rows(FAKE + 0x1000 * i)) for i, n in enumerate(("Q", "K", "V", "O"))}
    ws_bytes = o.get("ws_bytes", sa.sage_attn_packed_ws_bytes(*SHAPE.values(), False))
    t = {n: x and ctypes.byref(x) for n, x in t.items()}
    return sa.sage_attn_packed_fwd(t["Q"], t["K"], t["V"], o.get("cu", FAKE), t["O"], o.get("LSE", FAKE), o.get("ws", FAKE),
                                   ws_bytes, *s.values(), 1, o.get("sm_scale", 0.0), None)


def backward(**o):
    s = SHAPE | {n: o[n] for n in SHAPE if n in o}
    names = ("Q", "K", "V", "O", "dO", "dQ", "dK", "dV")
    t = {n: o.get(n, rows(FAKE + 0x1000 * (i + 1))) for i, n in enumerate(names)}
    ws_bytes = o.get("ws_bytes", sa.sage_attn_packed_ws_bytes(*SHAPE.values(), True))
    t = {n: x and ctypes.byref(x) for n, x in t.items()}
    return sa.sage_attn_packed_bwd(t["Q"], t["K"], t["V"], t["O"], o.get("LSE", FAKE), t["dO"], o.get("cu", FAKE), t["dQ"], t["dK"],
                                   t["dV"], o.get("ws", FAKE), ws_bytes, *s.values(), 1, o.get("sm_scale", 0.0), None)


BAD_SHAPES = [dict(T=0), dict(T=(1 << 24) + 1), dict(S=0), dict(S=65537), dict(H=0), dict(H=3), dict(Hkv=0), dict(Hkv=3),
              dict(H=258, Hkv=2), dict(H=65536, Hkv=65536), dict(D=96), dict(D=0), dict(D=256)]


@pytest.mark.parametrize("over", BAD_SHAPES, ids=str)
def test_shapes_outside_the_supported_set(lib, over):
    assert forward(**over) == sa.SAGE_ERR_UNSUPPORTED
    assert backward(**over) == sa.SAGE_ERR_UNSUPPORTED
    assert sa.sage_attn_packed_ws_bytes(*(SHAPE | over).values(), True) == 0


BAD_ROWS = [None, rows(p=None), rows(p=FAKE + 8), rows(token=0), rows(token=-512), rows(token=516), rows(head=0), rows(head=4),
            rows(head=-128), rows(token=1 << 38), rows(head=1 << 39)]
OVERLAPPING = [rows(token=64, head=512), rows(token=504, head=128), rows(token=512, head=120), rows(token=128, head=128 * 299)]


@pytest.mark.parametrize("bad", BAD_ROWS, ids=lambda r: "null" if r is None else f"{r.p}_{r.token}_{r.head}")
def test_rows_that_tma_does_not_take(lib, bad):
    bad = NULL_ROWS if bad is None else bad
    for n in ("Q", "K", "V", "O"):
        assert forward(**{n: bad}) == sa.SAGE_ERR_INVALID_ARG, n
        assert backward(**{n: bad}) == sa.SAGE_ERR_INVALID_ARG, n
    for n in ("dO", "dQ", "dK", "dV"):
        assert backward(**{n: bad}) == sa.SAGE_ERR_INVALID_ARG, n


@pytest.mark.parametrize("bad", OVERLAPPING, ids=lambda r: f"{r.token}_{r.head}")
def test_outputs_whose_rows_overlap(lib, bad):
    assert forward(O=bad) == sa.SAGE_ERR_INVALID_ARG
    for n in ("dQ", "dK", "dV"):
        assert backward(**{n: bad}) == sa.SAGE_ERR_INVALID_ARG, n


def test_other_bad_arguments(lib):
    for call in (forward, backward):
        for over in (dict(cu=None), dict(cu=FAKE + 2), dict(LSE=None), dict(LSE=FAKE + 1), dict(ws=None), dict(ws=FAKE + 128),
                     dict(ws_bytes=255), dict(sm_scale=math.nan), dict(sm_scale=math.inf)):
            assert call(**over) == sa.SAGE_ERR_INVALID_ARG, over
    # outputs over inputs or each other
    for n in ("Q", "K", "V"):
        assert forward(**{n: rows(FAKE + 0x3000)}) == sa.SAGE_ERR_INVALID_ARG
    for n in ("dQ", "dK", "dV"):
        for i in range(1, 6):
            assert backward(**{n: rows(FAKE + 0x1000 * i)}) == sa.SAGE_ERR_INVALID_ARG
    assert backward(dQ=rows(FAKE + 0x8000)) == sa.SAGE_ERR_INVALID_ARG
    assert backward(dK=rows(FAKE + 0x8000)) == sa.SAGE_ERR_INVALID_ARG


def test_workspaces(lib):
    for shape in ((1, 1, 1, 1, 64), (300, 3, 4, 2, 128), (1 << 20, 65536, 32, 8, 128), (1 << 24, 1, 1, 1, 64)):
        f, b = (sa.sage_attn_packed_ws_bytes(*shape, w) for w in (False, True))
        assert f >= 256 and f % 256 == 0 and b % 256 == 0 and b >= f + 8 * shape[0] * shape[2]


def heads(p=FAKE, batch=64 * 128, token=512, head=128):
    return sa.sage_heads(p, batch, token, head)


def turn(**o):
    r = sa.sage_rotary(o.get("turns", FAKE), o.get("rot", 64), 0, o.get("gain", 1.0))
    t = {n: o.get(n, heads(FAKE + 0x1000 * i)) for i, n in enumerate(("Q", "Qo", "K", "Ko"))}
    t = {n: x and ctypes.byref(x) for n, x in t.items()}
    a = dict(positions=None, start=FAKE, cu=None, B=2, N=16, S=0, H=4, Hkv=2, D=128)
    a |= {n: o[n] for n in a if n in o}
    return sa.sage_attn_rotary(NULL if o.get("null") else r, *t.values(), *a.values(), 0, None)


NULL = ctypes.POINTER(sa.sage_rotary)()


def test_rotary_refuses(lib):
    for over in (dict(null=True), dict(turns=None), dict(turns=FAKE + 4), dict(gain=math.nan), dict(gain=math.inf), dict(Q=NULL_HEADS),
                 dict(Qo=NULL_HEADS), dict(K=NULL_HEADS), dict(Ko=NULL_HEADS), dict(Q=heads(FAKE + 8)), dict(K=heads(token=4)),
                 dict(Qo=heads(0x90000, head=64)), dict(Qo=heads(0x90000, batch=512)), dict(Ko=heads(0x90000, token=0)),
                 dict(Qo=heads(FAKE, token=1024, batch=64 * 1024)), dict(Qo=heads(FAKE + 0x2000)), dict(Ko=heads(FAKE)),
                 dict(Ko=heads(FAKE + 0x1000)), dict(positions=FAKE), dict(positions=FAKE + 2, start=None), dict(start=FAKE + 1),
                 dict(cu=FAKE, S=2), dict(positions=FAKE, start=None, cu=FAKE, S=2, B=1), dict(cu=FAKE + 2, S=2, B=1)):
        assert turn(**over) == sa.SAGE_ERR_INVALID_ARG, over
    for over in (dict(D=96), dict(rot=0), dict(rot=24), dict(rot=144), dict(rot=128, D=64), dict(B=0), dict(N=0), dict(H=0),
                 dict(H=32768), dict(Hkv=0), dict(B=1 << 16, N=1 << 15), dict(cu=FAKE, S=0, B=1)):
        assert turn(**over) == sa.SAGE_ERR_UNSUPPORTED, over


def test_helpers_check_their_tensors(lib):
    q, k, cu = torch.zeros(8, 2, 64, dtype=torch.bfloat16), torch.zeros(8, 1, 64, dtype=torch.bfloat16), torch.tensor([0, 8])
    for bad in ((q[0], k, k, cu), (q, k[0], k, cu), (q, k, k, cu[:1]), (q, k, k, cu[None])):
        with pytest.raises(ValueError):
            sa.packed_forward(*bad)
    with pytest.raises(ValueError, match="GPU"):
        sa.packed_forward(q, k, k, cu)
    with pytest.raises(sa.SageError):
        sa.alloc_packed_ws(8, 1, 3, 2, 64)
    for kw in (dict(rot=24), dict(rot=0), dict(rot=144)):
        with pytest.raises(sa.SageError):
            sa.rotary_table(**kw, device="cpu")
    for kw in (dict(rot=64, scaling="other"), dict(rot=64, base=1.0), dict(rot=64, factor=0.5), dict(rot=64, frequencies=[1.0]),
               dict(rot=64, scaling="ramp", factor=2.0, fast=1.0), dict(rot=64, frequencies=[math.nan] * 32)):
        with pytest.raises(ValueError):
            sa.rotary_table(**kw, device="cpu")
    for kw in (dict(turns=torch.zeros(32)), dict(turns=torch.zeros((2, 8), dtype=torch.int64)), dict(turns=torch.zeros(32, dtype=torch.int64))):
        with pytest.raises(ValueError):
            sa.Rotary(**kw)


def test_frequencies():
    f, gain = sa.rotary_frequencies(64)
    assert gain == 1.0 and f[0] == 1.0 and f[-1] == pytest.approx(10000.0 ** (-62 / 64), rel=1e-14)
    assert all(x > y for x, y in zip(f, f[1:]))
    assert sa.rotary_frequencies(64, scaling="linear", factor=4.0) == ([x / 4.0 for x in f], 1.0)
    g, gain = sa.rotary_frequencies(64, scaling="base", factor=4.0)
    assert gain == 1.0 and g[0] == 1.0 and g[-1] == pytest.approx(f[-1] / 4.0, rel=1e-12)
    g, gain = sa.rotary_frequencies(64, scaling="ramp", factor=4.0, context=4096)
    assert gain == pytest.approx(0.1 * math.log(4.0) + 1.0)
    for x, y in zip(f, g):
        turns = x * 4096 / (2 * math.pi)
        assert x / 4.0 <= y * (1 + 1e-12) and y <= x * (1 + 1e-12)
        assert turns <= 40.0 or y == pytest.approx(x)          # (a pair beyond the borders, which lie on whole pairs)
        assert turns >= 0.75 or y == pytest.approx(x / 4.0)
    assert sa.rotary_frequencies(64, scaling="ramp", factor=1.0) == (pytest.approx(f), 1.0)
