"""The paged cache without a GPU: its entry points refuse bad arguments before anything is
launched, its workspaces have their sizes, the torch helpers check their tensors, and the numpy
reference of the GPU tests is itself checked (rounding of the codes against torch's casts, a
closed-form attention)."""
import functools
import ctypes

import numpy as np
import pytest
import torch

import bit_trainable_attention_sagebwd_gb300 as sa
import kv_ref


@pytest.fixture(scope="module")
def lib():
    from bit_trainable_attention_sagebwd_gb300 import build
    build.build()
    return sa.lib()


FAKE = 0x10000  # aligned, never dereferenced: the checks fail first


def cache(**over):
    v = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, table=FAKE, lengths=FAKE, refs=FAKE, status=FAKE, n_pages=8,
             Hkv=2, page=64, D=128, n_slots=4, max_pages=8, kind=0)
    return sa.sage_kv_cache(**(v | over))


def calls(c, to=None):
    """Every call on the cache c, with arguments that are otherwise good."""
    n = sa.sage_attn_kv_ws_bytes(4, 4, 2, 128, 1)
    w = sa.sage_attn_kv_compact_ws_bytes(8)
    other = {k: 0x900000 for k in ("k", "v", "k_scale", "v_scale", "table", "lengths", "refs")}
    to = cache(**other) if to is None else to
    return {
        "append": lambda **o: sa.sage_attn_kv_append(c, *({k: o.get(k, FAKE) for k in ("K", "V", "shift", "slots", "pos", "n_new")}).values(),
                                                     o.get("B", 4), o.get("Nn", 5), None),
        "attention": lambda **o: sa.sage_attn_kv_attention(c, *({k: o.get(k, FAKE) for k in ("Q", "slots", "q_len", "O", "LSE", "ws")}).values(),
                                                           o.get("ws_bytes", n), o.get("B", 4), o.get("H", 4), o.get("Nq", 1), 1,
                                                           o.get("sm_scale", 0.0), None),
        "fork": lambda **o: sa.sage_attn_kv_fork(c, o.get("src", FAKE), None),
        "extend": lambda **o: sa.sage_attn_kv_extend(c, o.get("n_new", FAKE), o.get("pos", FAKE), o.get("cow", FAKE), None),
        "truncate": lambda **o: sa.sage_attn_kv_truncate(c, o.get("keep", FAKE), None),
        "compact": lambda **o: sa.sage_attn_kv_compact(c, to, o.get("ws", FAKE), o.get("ws_bytes", w), None),
    }


BAD_CACHE = [(dict(k=None), 1), (dict(v=FAKE + 8), 1), (dict(k_scale=FAKE + 2), 1), (dict(v_scale=None), 1),
             (dict(table=FAKE + 1), 1), (dict(lengths=None), 1), (dict(refs=FAKE + 4), 1), (dict(status=None), 1),
             (dict(page=48), 2), (dict(page=0), 2), (dict(page=256), 2), (dict(D=96), 2), (dict(kind=2), 2),
             (dict(Hkv=0), 2), (dict(n_pages=0), 2), (dict(n_slots=0), 2), (dict(n_slots=8193), 2),
             (dict(max_pages=0), 2), (dict(max_pages=1 << 26, page=128), 2)]


@pytest.mark.parametrize("over,code", BAD_CACHE, ids=[str(b[0]) for b in BAD_CACHE])
def test_a_bad_cache_is_refused_by_every_call(lib, over, code):
    for name, call in calls(cache(**over)).items():
        assert call() == code, name
    null = ctypes.POINTER(sa.sage_kv_cache)()
    for name, call in calls(null).items():
        assert call() == sa.SAGE_ERR_INVALID_ARG, name


def test_bad_arguments_are_refused(lib):
    c = calls(cache())
    odd = FAKE + 2
    for name in ("K", "V", "pos", "n_new"):
        assert c["append"](**{name: None}) == sa.SAGE_ERR_INVALID_ARG
    for name in ("K", "V", "shift", "slots", "pos", "n_new"):
        assert c["append"](**{name: odd}) == sa.SAGE_ERR_INVALID_ARG
    assert c["append"](slots=None, B=5) == sa.SAGE_ERR_INVALID_ARG  # more rows than slots
    for over in (dict(B=0), dict(Nn=0), dict(B=65536)):
        assert c["append"](**over) == sa.SAGE_ERR_UNSUPPORTED
    for name in ("Q", "O", "LSE", "ws"):
        assert c["attention"](**{name: None}) == sa.SAGE_ERR_INVALID_ARG
    for name in ("Q", "slots", "q_len", "O", "LSE", "ws"):
        assert c["attention"](**{name: odd}) == sa.SAGE_ERR_INVALID_ARG
    for scale in (float("nan"), float("inf")):
        assert c["attention"](sm_scale=scale) == sa.SAGE_ERR_INVALID_ARG
    assert c["attention"](slots=None, B=5, ws_bytes=1 << 40) == sa.SAGE_ERR_INVALID_ARG
    assert c["attention"](ws_bytes=sa.sage_attn_kv_ws_bytes(4, 4, 2, 128, 1) - 1) == sa.SAGE_ERR_INVALID_ARG
    for over in (dict(H=3), dict(H=0), dict(B=0), dict(B=4097), dict(Nq=0)):
        assert c["attention"](**over) == sa.SAGE_ERR_UNSUPPORTED
    for call, names in (("fork", ["src"]), ("extend", ["n_new", "pos", "cow"]), ("truncate", ["keep"])):
        for name in names:
            for bad in (None, odd):
                assert c[call](**{name: bad}) == sa.SAGE_ERR_INVALID_ARG
    a, b = FAKE + 0x1000, FAKE + 0x2000
    for over in (dict(n_new=a, pos=a, cow=b), dict(n_new=a, pos=b, cow=a), dict(n_new=a, pos=b, cow=b)):
        assert c["extend"](**over) == sa.SAGE_ERR_INVALID_ARG
    assert c["attention"](O=FAKE, Q=FAKE) == sa.SAGE_ERR_INVALID_ARG
    assert c["compact"](ws=None) == sa.SAGE_ERR_INVALID_ARG
    assert c["compact"](ws_bytes=sa.sage_attn_kv_compact_ws_bytes(8) - 1) == sa.SAGE_ERR_INVALID_ARG
    assert calls(cache(), to=cache())["compact"]() == sa.SAGE_ERR_INVALID_ARG  # into itself
    far = {k: 0x900000 for k in ("k", "v", "k_scale", "v_scale", "table", "lengths", "refs")}
    for over in (dict(page=32), dict(D=64), dict(Hkv=1), dict(kind=1), dict(n_slots=3), dict(max_pages=7)):
        assert calls(cache(), to=cache(**(far | over)))["compact"]() == sa.SAGE_ERR_INVALID_ARG
    assert sa.status_str(sa.SAGE_ERR_NO_PAGES) == "too few free pages"


def test_workspace_sizes(lib):
    for bad in [(0, 4, 2, 128, 1), (4097, 4, 2, 128, 1), (1, 3, 2, 128, 1), (1, 4, 2, 96, 1), (1, 4, 2, 128, 0),
                (4096, 1 << 20, 1 << 14, 128, 1 << 20)]:
        assert sa.sage_attn_kv_ws_bytes(*bad) == 0
    for ok in [(1, 1, 1, 64, 1), (4096, 32, 8, 128, 1), (1, 32, 1, 128, 2048), (7, 15, 3, 64, 33)]:
        n = sa.sage_attn_kv_ws_bytes(*ok)
        assert 0 < n < 1 << 30
    assert sa.sage_attn_kv_compact_ws_bytes(0) == 0
    assert sa.sage_attn_kv_compact_ws_bytes(100) >= 256 + 800


def test_helpers_check_their_tensors():
    z = functools.partial(torch.zeros, dtype=torch.float32)
    good = dict(k=z((4, 2, 64, 128), dtype=torch.int8), v=z((4, 2, 64, 128), dtype=torch.int8), k_scale=z((4, 2)),
                v_scale=z((4, 2)), table=z((3, 5), dtype=torch.int32), lengths=z(3, dtype=torch.int32),
                refs=z(4, dtype=torch.int32), status=z(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        sa.KVCache(**good)
    with pytest.raises(ValueError):
        sa.KVCache(**(good | dict(k=z((4, 2, 64, 128)))))
    with pytest.raises(ValueError):
        sa.kv_cache(4, 2, 128, 3, 5, kind="fp4")
    for bad in (dict(page=48), dict(d=96), dict(n_pages=0)):
        with pytest.raises(sa.SageError):
            sa.kv_cache(**(dict(n_pages=4, hkv=2, d=128, n_slots=3, max_pages=5) | bad))
    from bit_trainable_attention_sagebwd_gb300 import kvcache
    t = z((2, 3))
    cpu = torch.device("cpu")
    assert kvcache._arg(t, "t", torch.float32, (2, 3), cpu) == t.data_ptr()
    for args in ((t, "t", torch.int32, (2, 3), cpu), (t, "t", torch.float32, (3, 2), cpu),
                 (t, "t", torch.float32, (2, 3), torch.device("cuda", 0)), (t.T, "t", torch.float32, (3, 2), cpu)):
        with pytest.raises(ValueError):
            kvcache._arg(*args)


def test_reference_codes():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(0, 100, 20000), rng.uniform(-2 ** -6, 2 ** -6, 5000), kv_ref.E4M3[:127], [-0.0, 1e-9]])
    x = np.clip(x, -448, 448).astype(np.float32)
    mid = ((kv_ref.E4M3[:126] + kv_ref.E4M3[1:127]) / 2).astype(np.float32)
    x = np.concatenate([x, mid, -mid])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv_ref.encode(x, "e4m3"), want)
    b = np.arange(256, dtype=np.uint8)
    finite = (b & 127) != 127
    assert np.array_equal(kv_ref.decode(b, "e4m3")[finite], torch.from_numpy(b).view(torch.float8_e4m3fn).double().numpy()[finite])
    assert np.array_equal(kv_ref.encode(np.float32([0.5, 1.5, -2.5, 126.6, -127.2]), "int8").view(np.int8), [0, 2, -2, 127, -127])


def test_reference_attention_closed_form():
    """Equal keys: O is the mean of the values seen, LSE = S + log n; without keys 0 and -inf."""
    c = kv_ref.Cache(4, 1, 64, 2, 4, 16, "int8")
    pos, _ = c.extend([20, 0])
    k = np.ones((2, 1, 20, 64), np.float32)
    v = np.repeat(np.arange(1, 21, dtype=np.float32)[None, None, :, None], 64, 3).repeat(2, 0)
    c.append(k, v, pos, [20, 0])
    q = np.full((2, 1, 2, 64), 0.25)
    o, lse, *_ = c.attention(q)
    _, vals = c.values(0, 0)
    assert np.allclose(o[0, 0, 1], vals.mean(0)) and np.allclose(o[0, 0, 0], vals[:19].mean(0))
    assert np.allclose(lse[0, 0], 2.0 + np.log([19, 20])) and np.all(lse[1] == -np.inf) and not o[1].any()


def test_the_selftest_of_the_join_refuses_bad_arguments(lib):
    n = sa.sage_attn_kv_ws_bytes(4, 4, 2, 128, 1)

    def call(c=None, O=FAKE, LSE=FAKE, ws=FAKE, ws_bytes=n, B=4, H=4, Nq=1):
        return sa.sage_attn_selftest_kv_join(cache() if c is None else c, O, LSE, ws, ws_bytes, B, H, Nq, None)

    for over in (dict(O=None), dict(O=FAKE + 8), dict(LSE=None), dict(ws=None), dict(ws_bytes=n - 1), dict(c=cache(k=None))):
        assert call(**over) == sa.SAGE_ERR_INVALID_ARG
    for over in (dict(B=0), dict(H=3), dict(Nq=0), dict(c=cache(D=96))):
        assert call(**over) == sa.SAGE_ERR_UNSUPPORTED


# ------------------------------------------------------------------------------ what the formats cost

def stored(kind, page, n, step, seed, d=64):
    """Keys and values, each page's tokens of a size of their own that rises and falls, written `step` tokens at a
    time: the cache, the bf16 values, and for each token and head the scales of its page since it was written."""
    rng = np.random.default_rng(seed)
    c = kv_ref.Cache(-(-n // page), 2, d, 1, -(-n // page), page, kind)
    size = np.exp(rng.uniform(-2, 2, (1, 1, n, 1)))
    k, v = (torch.from_numpy((rng.standard_normal((1, 2, n, d)) * size).astype(np.float32)).to(torch.bfloat16).float().numpy()
            for _ in range(2))
    since = np.zeros((2, 2, n, n), np.float32)  # [K or V, head, token, write]: the page's scale after it, 0: not yet there
    at = 0
    while at < n:
        m = min(step, n - at)
        pos, _ = c.extend([m])
        c.append(k[:, :, at:at + m], v[:, :, at:at + m], pos, [m])
        pages = c.table[0, np.arange(at + m) // page]
        since[0, :, :at + m, at], since[1, :, :at + m, at] = c.k_scale[pages].T, c.v_scale[pages].T
        at += m
    return c, k[0], v[0], since


def rounding(kind, x, since):
    """How far a stored value may be from x: half a step of its code at each scale that its page has had since
    (the code is rounded anew only where the scale changes), and fp32's roundings of scale, quotient and product.  int8: a
    step is the scale; e4m3: 2^-3 of the value down to 2^-6 of the unit, below it 2^-9 of the scale."""
    changed = np.concatenate((since[..., :1] > 0, (since[..., 1:] != since[..., :-1])), -1)
    s = np.where(changed, since, 0).astype(np.float64)[:, :, None, :]       # [head, token, 1, write]
    bound = np.zeros(x.shape)
    for w in range(s.shape[-1]):
        half = 0.5 * s[..., w] if kind == "int8" else np.where(s[..., w] > 0, np.maximum(2.0 ** -4 * (np.abs(x) + bound), 2.0 ** -10 * s[..., w]), 0)
        bound += half + 2.0 ** -22 * np.where(s[..., w] > 0, np.abs(x) + bound, 0)
    return bound


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("step", [1, 7, 100])
def test_stored_values_are_within_the_formats_rounding(kind, page, step):
    """One write of a prompt is off by half a step; token by token each growth of the page's scale adds another
    half step, and the scales end up the same."""
    n = 100
    c, k, v, since = stored(kind, page, n, step, page + step)
    once, *_ = stored(kind, page, n, n, page + step)
    pages = [np.arange(n) // page]
    for h in range(2):
        for x, got, was in zip((k, v), c.values(0, h), since):
            bound = rounding(kind, x, was)[h]
            assert np.all(np.abs(got - x[h]) <= bound)
            if step == n:  # the definition: no value of a page needs a larger step
                top = np.array([np.abs(x[h][pages[0] == p]).max() for p in pages[0]])
                worst = top / 254 if kind == "int8" else np.maximum(2.0 ** -4 * np.abs(x[h]).max(1), top / 448 * 2.0 ** -10)
                # (int8: |x| is up to 127 steps, so 2^-22 |x| is up to 254 x 2^-22 < 2^-14 of half a step)
                assert np.all(bound.max(1) <= worst * (1 + 2.0 ** -13))
    assert np.array_equal(c.k_scale, once.k_scale) and np.array_equal(c.v_scale, once.v_scale)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("step", [1, 100])
def test_attention_over_stored_values_against_the_keys_themselves(kind, step):
    """Every logit is off by sm_scale sum |q| dk at most, dk the stored key's rounding; weights by e to twice the
    largest of these, O by that and by the values' own rounding."""
    rng = np.random.default_rng(step)
    n, d = 100, 64
    c, k, v, since = stored(kind, 64, n, step, 5, d)
    dk, dv = rounding(kind, k, since[0]), rounding(kind, v, since[1])
    q = rng.standard_normal((1, 2, 1, d)) * 0.2
    o, lse, *_ = c.attention(q)
    for h in range(2):
        t = k[h] @ q[0, h, 0] / np.sqrt(d)
        far = (dk[h] @ np.abs(q[0, h, 0])).max() / np.sqrt(d)
        p = np.exp(t - t.max())
        p /= p.sum()
        bound = (np.exp(2 * far) - 1) * (p @ np.abs(v[h])) + np.exp(2 * far) * (p @ dv[h])
        assert np.all(np.abs(o[0, h, 0] - p @ v[h]) <= bound)
        assert abs(lse[0, h, 0] - (t.max() + np.log(np.exp(t - t.max()).sum()))) <= far
