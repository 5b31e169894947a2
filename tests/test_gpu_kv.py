"""The 8-bit paged cache on the GPU (sage_attn_kv_*) against its plain numpy form (kv_ref.py):
codes, scales, tables, lengths and refs bit for bit, attention within the roundings that its
definition names (kv_ref.attention_tolerances)."""
import threading

import numpy as np
import pytest
import torch

import bit_trainable_attention_sagebwd_gb300 as sa
import kv_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def fp32_default():
    """torch's default type as it is for a user: another module of the run may have changed it."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


def bf16(rng, shape, scale=1.0):
    """Values on the GPU in bf16, and the same as fp32 on the host."""
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)
    return t.cuda(), t.float().numpy()


def pair(n_pages, hkv, d, n_slots, max_pages, page, kind, poison=True):
    """An empty cache on the GPU and its reference.  Free memory holds what earlier use may leave
    there: the largest codes, NaN in e4m3 among them, NaN scales and page numbers out of range."""
    c = sa.kv_cache(n_pages, hkv, d, n_slots, max_pages, page=page, kind=kind)
    r = kv_ref.Cache(n_pages, hkv, d, n_slots, max_pages, page, kind)
    if poison:
        for a, b in ((c.k, r.k), (c.v, r.v)):
            a.view(torch.int8).fill_(127)
            b[:] = 127
        for a, b in ((c.k_scale, r.k_scale), (c.v_scale, r.v_scale)):
            a.fill_(float("nan"))
            b[:] = np.nan
        c.table.fill_(-2 ** 31)
        r.table[:] = -2 ** 31
    return c, r


def same_state(c, r):
    torch.cuda.synchronize()
    assert np.array_equal(c.lengths.cpu().numpy(), r.lengths)
    assert np.array_equal(c.refs.cpu().numpy(), r.refs)
    for s, n in enumerate(r.lengths):
        m = r.pages(int(n))
        assert np.array_equal(c.table[s, :m].cpu().numpy(), r.table[s, :m]), f"table of slot {s}"
    for name in ("k", "v"):
        got, want = getattr(c, name).view(torch.uint8).cpu().numpy(), getattr(r, name)
        assert np.array_equal(got, want), f"{name}: {np.sum(got != want)} codes differ"
        assert np.array_equal(getattr(c, name + "_scale").cpu().numpy(), getattr(r, name + "_scale"), equal_nan=True)


def fill(c, r, rng, lengths, shift=None, step=None):
    """Append `lengths` tokens to the slots, at most `step` at a time."""
    left = np.asarray(lengths)
    step = step or max(1, int(left.max(initial=1)))
    while left.any():
        n = np.minimum(left, step)
        pos = sa.kv_extend(c, dev(n))
        rpos, _ = r.extend(n)
        assert np.array_equal(pos.cpu().numpy(), rpos)
        shape = (len(left), r.k.shape[1], int(n.max()), r.k.shape[3])
        k, kf = bf16(rng, shape, 1.5)
        v, vf = bf16(rng, shape)
        sa.kv_append(c, k, v, pos, dev(n), k_shift=None if shift is None else dev(shift, torch.float32))
        r.append(kf, vf, rpos, n, shift=shift)
        left = left - n


def check_attention(c, r, rng, H, Nq, causal=True, slots=None, q_len=None, sm_scale=None, q_scale=1.0, **kw):
    B = c.n_slots if slots is None else len(slots)
    q, qf = bf16(rng, (B, H, Nq, c.d), q_scale)
    o = torch.full((B, H, Nq, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H, Nq), 7.0, device="cuda")
    sa.kv_attention(q, c, causal=causal, slots=None if slots is None else dev(slots), q_len=None if q_len is None else dev(q_len),
                    sm_scale=sm_scale, o=o, lse=lse, **kw)
    torch.cuda.synchronize()
    assert sa.get_status(c.status) == sa.SAGE_OK
    compare(o, lse, r.attention(qf.astype(np.float64), causal, slots, q_len, sm_scale), int(r.lengths.max(initial=0)), c.d)
    return q, o, lse


def compare(o, lse, want, n, d):
    wo, wl, pv, av, mag, rows = want
    tol_o, tol_l = kv_ref.attention_tolerances(wo, wl, pv, av, mag, n, d)
    go, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(go[~rows] == 7.0) and np.all(gl[~rows] == 7.0), "rows behind q_len were written"
    empty = rows & (wl == -np.inf)
    assert np.all(go[empty] == 0.0) and np.all(gl[empty] == -np.inf)
    full = rows & ~empty
    eo, el = np.abs(go[full] - wo[full]), np.abs(gl[full] - wl[full])
    assert np.all(eo <= tol_o[full]), f"O off by up to {np.max(eo / tol_o[full]):.3g} of its tolerance"
    assert np.all(el <= tol_l[full]), f"LSE off by up to {np.max(el / tol_l[full]):.3g} of its tolerance"


# ------------------------------------------------------------------------------ append

@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("page,d", [(16, 64), (16, 128), (32, 128), (64, 64), (64, 128), (128, 64), (128, 128)])
def test_append_codes(kind, page, d):
    """Prompts of odd lengths, then tokens one and a few at a time (pages begun before, whose scale
    grows or stays), with and without a shift of the keys: bit for bit."""
    rng = np.random.default_rng(page + d)
    c, r = pair(40, 3, d, 4, 20, page, kind)
    shift = rng.standard_normal((3, d)).astype(np.float32)
    fill(c, r, rng, [0, 1, page - 1, page + 1], shift)
    same_state(c, r)
    fill(c, r, rng, [5, 0, 2, 3], shift, step=1)
    same_state(c, r)
    fill(c, r, rng, [2 * page + 3, 1, page, 0])
    same_state(c, r)
    assert sa.get_status(c.status) == sa.SAGE_OK


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_append_extreme_values(kind):
    """Blocks of zeros (scale 0), the largest and the smallest bf16 (subnormal scales), a page whose
    scale grows by 2^60, and quotients that fall on rounding borders."""
    c, r = pair(8, 1, 64, 1, 8, 16, kind, poison=False)
    rng = np.random.default_rng(5)
    big = float(torch.finfo(torch.bfloat16).max)
    steps = [np.zeros((3, 64)), np.full((2, 64), 2.0 ** -133), np.full((1, 64), 2.0 ** -70), rng.standard_normal((4, 64)),
             np.where(rng.random((16, 64)) < 0.5, big, -big), np.arange(-32, 32)[None].repeat(3, 0) * 0.5,
             np.full((3, 64), 2.0 ** -130), rng.standard_normal((9, 64)) * 2.0 ** -126]
    for x in steps:
        k = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)[None, None]
        n = dev([x.shape[0]])
        pos = sa.kv_extend(c, n)
        rpos, _ = r.extend([x.shape[0]])
        sa.kv_append(c, k.cuda(), (-k).cuda().contiguous(), pos, n)
        r.append(k.float().numpy(), -k.float().numpy(), rpos, [x.shape[0]])
        same_state(c, r)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("top", [60, 100, 190, 700, 2000, 40000])
def test_append_saturates_where_the_scale_is_subnormal(top, kind):
    """Keys that a shift leaves at `top` units of 2^-149, below what their bf16 form can be: the scale has one or a
    few bits, quotients pass the largest code and saturate.  Tokens that let the scale grow follow."""
    rng = np.random.default_rng(14)
    c, r = pair(4, 2, 64, 1, 4, 16, kind, poison=False)
    v = torch.zeros((1, 2, 5, 64), dtype=torch.bfloat16)
    for grow in (1, 3, 2 ** 20):
        units = rng.integers(-top, top + 1, (2, 64))
        units[:, 0], units[:, 1] = top, -top
        shift = np.float32(units * grow * 2.0 ** -149)
        pos = sa.kv_extend(c, dev([5]))
        rpos, _ = r.extend([5])
        sa.kv_append(c, v.cuda(), v.cuda(), pos, dev([5]), k_shift=dev(shift, torch.float32))
        r.append(v.float().numpy(), v.float().numpy(), rpos, [5], shift=shift)
        same_state(c, r)


def test_append_slots_and_padding():
    """Rows that belong to other slots, rows without tokens, NaN behind the tokens that count."""
    rng = np.random.default_rng(11)
    c, r = pair(30, 2, 64, 5, 8, 16, "int8")
    n = np.array([3, 0, 17, 1, 9])
    pos, (rpos, _) = sa.kv_extend(c, dev(n)), r.extend(n)
    slots = [4, 2, 0]
    k, kf = bf16(rng, (3, 2, 20, 64))
    v, vf = bf16(rng, (3, 2, 20, 64))
    for b, s in enumerate(slots):
        k[b, :, n[s]:] = float("nan")
        v[b, :, n[s]:] = float("inf")
    sa.kv_append(c, k, v, pos, dev(n), slots=dev(slots))
    r.append(kf, vf, rpos, n, slots=slots)
    same_state(c, r)
    assert sa.get_status(c.status) == sa.SAGE_OK


def test_append_leaves_out_what_it_must_not_write():
    rng = np.random.default_rng(12)
    c, r = pair(30, 2, 64, 4, 4, 16, "int8")
    fill(c, r, rng, [10, 20, 0, 0])
    k, kf = bf16(rng, (4, 2, 4, 64))

    def refused(pos, n, slots=None):
        sa.kv_append(c, k, k, dev(pos), dev(n), slots=None if slots is None else dev(slots))
        same_state(c, r)
        assert sa.get_status(c.status) == sa.SAGE_ERR_INVALID_ARG
        assert sa.get_status(c.status) == sa.SAGE_OK  # read and cleared

    refused([0, 0, 0, 0], [0, 0, 2, 0])                      # slot 2 has no pages (its table is out of range)
    refused([0, 63, 0, 0], [0, 4, 0, 0])                     # past the reserved pages and the table
    refused([0, 0, 0, 0], [5, 0, 0, 0])                      # more tokens than K and V hold
    refused([2 ** 31 - 8, 0, 0, 0], [4, 0, 0, 0])
    refused([8, 0, 0, 0], [0, 0, 0, 0], [4, -1, 1, 0])       # slots that are not there
    refused([2 ** 31 - 2, 0, 0, 0], [4, 0, 0, 0])            # tokens on both sides of 2^31
    sa.kv_fork(c, dev([-1, -1, 0, -1]))                      # slots 0 and 2 share a page
    r.fork([-1, -1, 0, -1])
    refused([8, 0, 0, 0], [2, 0, 0, 0])
    # a slot named twice: the first row counts
    sa.kv_append(c, k, k, dev([0, 18, 0, 0]), dev([0, 2, 0, 0]), slots=dev([0, 1, 1, 2]))
    r.append(kf[1:2], kf[1:2], [0, 18, 0, 0], [0, 2, 0, 0], slots=[1])
    same_state(c, r)
    assert sa.get_status(c.status) == sa.SAGE_ERR_INVALID_ARG


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [16, 64])
def test_append_behind_the_length_of_a_slot(page, kind):
    """What a table lists behind its slot's length may be another slot's page: tokens that were not given
    room are not written, wherever the old entries point."""
    rng = np.random.default_rng(17)
    c, r = pair(12, 2, 64, 4, 6, page, kind, poison=False)  # (tables of zeros: page 0 everywhere)
    fill(c, r, rng, [2 * page + 3, 0, 0, 0])
    k, _ = bf16(rng, (4, 2, 2 * page, 64), 50.0)

    def refused(pos, n, slots=None):
        sa.kv_append(c, k, k, dev(pos), dev(n), slots=None if slots is None else dev(slots))
        same_state(c, r)
        assert sa.get_status(c.status) == sa.SAGE_ERR_INVALID_ARG

    refused([-1, 0, -1, -1], [0, 3, 0, 0])                   # slot 1 was not extended; its table says page 0
    refused([-1, 0, 0, 0], [0, page, 1, page + 1])           # three such slots
    refused([-1, 0, 0, 0], [0, 5, 5, 5], [2, 1, 3, 0])       # rows of other slots
    fill(c, r, rng, [0, page + 2, 0, 0])
    sa.kv_truncate(c, dev([-1, 4, -1, -1]))                  # slot 1 gives its second page back, slot 2 takes it
    r.truncate([-1, 4, -1, -1])
    fill(c, r, rng, [0, 0, page, 0])
    assert r.table[1, 1] == r.table[2, 0]
    refused([-1, page, -1, -1], [0, 2, 0, 0])                # slot 1 at its old place
    refused([-1, 4, -1, -1], [0, page, 0, 0])                # from its last token on, across the end
    n = [0, 3, 0, 0]
    pos, (rpos, _) = sa.kv_extend(c, dev(n)), r.extend(n)
    refused(rpos, [0, page, 0, 0])                           # more than it was extended by
    k, kf = bf16(rng, (4, 2, 3, 64))
    sa.kv_append(c, k, k, pos, dev(n))
    r.append(kf, kf, rpos, n)
    same_state(c, r)
    assert sa.get_status(c.status) == sa.SAGE_OK


# ------------------------------------------------------------------------------ attention

@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attention_one_token(kind, d, page):
    """Lengths of nothing, one, around a chunk of 16 and a page, and of several parts."""
    rng = np.random.default_rng(page * d)
    lengths = [0, 1, 15, 16, 17, page - 1, page, page + 1, 333, 700]
    c, r = pair(200, 2, d, len(lengths), 60, page, kind)
    fill(c, r, rng, lengths)
    check_attention(c, r, rng, 8, 1)


GROUPS = [(1, 1, 1), (1, 7, 1), (2, 8, 1), (3, 5, 2), (1, 16, 1), (1, 32, 1), (2, 3, 7), (2, 1, 16), (1, 4, 33), (2, 2, 70),
          (1, 8, 130)]


@pytest.mark.parametrize("hkv,g,nq", GROUPS)
@pytest.mark.parametrize("d,kind", [(64, "e4m3"), (128, "int8"), (128, "e4m3")])
def test_attention_groups_and_queries(hkv, g, nq, d, kind):
    """Shared heads and several queries; slots in another order and twice, ragged q_len, more queries
    than keys (rows that see nothing), causal and not."""
    rng = np.random.default_rng(hkv + 10 * g + 100 * nq)
    c, r = pair(60, hkv, d, 5, 10, 64, kind)
    fill(c, r, rng, [130, 5, 0, 77, 200])
    slots, q_len = [3, 0, 4, 1, 2, 0], [nq, max(1, nq - 1), (nq + 1) // 2, nq, nq, 0]
    check_attention(c, r, rng, hkv * g, nq, True, slots, q_len)
    check_attention(c, r, rng, hkv * g, nq, False, slots[:4], None, sm_scale=0.3)


@pytest.mark.parametrize("g,nq", [(33, 1), (100, 2), (128, 1), (300, 1), (257, 3)])
@pytest.mark.parametrize("page,d,kind", [(16, 128, "e4m3"), (128, 64, "int8")])
def test_attention_groups_wider_than_a_row_tile(page, d, kind, g, nq):
    """One key/value head for so many query heads that a token's rows fill a unit, or lie in several."""
    rng = np.random.default_rng(g + page)
    c, r = pair(700 // page + 8, 1, d, 3, 500 // page + 1, page, kind)
    fill(c, r, rng, [333, 1, 64])
    check_attention(c, r, rng, g, nq, True, [2, 0, 1, 0], [nq, max(1, nq - 1), nq, 0])
    check_attention(c, r, rng, g, nq, False)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_attention_long(kind):
    """One sequence of 20,011 tokens among short ones: cut over the whole GPU."""
    rng = np.random.default_rng(3)
    c, r = pair(700, 1, 128, 3, 400, 64, kind)
    fill(c, r, rng, [20011, 1, 260])
    check_attention(c, r, rng, 4, 1)
    check_attention(c, r, rng, 4, 3, slots=[0, 2])


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_sharp_and_wide_values(nq):
    """Logits of hundreds (one key takes all), tiny and huge queries (their products stay in range
    after the row's power of two), pages whose V scales differ by 2^40."""
    rng = np.random.default_rng(8)
    c, r = pair(20, 1, 128, 2, 10, 16, "int8")
    fill(c, r, rng, [100, 37], step=16)
    for p in range(20):
        f = np.float32(2.0 ** ((p % 5) * 10 - 20))
        c.v_scale[p] *= float(f)
        r.v_scale[p] *= f
    for q_scale, sm_scale in ((60.0, None), (2.0 ** -100, 2.0 ** 98), (2.0 ** 100, 2.0 ** -102), (0.0, None)):
        check_attention(c, r, rng, 4, nq, sm_scale=sm_scale, q_scale=q_scale)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("nq", [1, 40])
def test_attention_logits_past_fp32_resolution(nq, kind):
    """Logits of 10^9 and more: which key wins is beyond fp32, but every output is a mean of values."""
    rng = np.random.default_rng(13)
    c, r = pair(20, 2, 128, 2, 10, 64, kind)
    fill(c, r, rng, [300, 77])
    q, _ = bf16(rng, (2, 4, nq, 128), 1e4)
    for sm_scale in (1e3, 1e5, 1e8, 1e12, 1e20):
        o, lse = sa.kv_attention(q, c, sm_scale=sm_scale)
        torch.cuda.synchronize()
        assert sa.get_status(c.status) == sa.SAGE_OK
        most = max(np.abs(r.values(s, h)[1]).max() for s in range(2) for h in range(2))
        assert torch.isfinite(o).all() and float(o.abs().max()) <= most * (1 + 2 ** -7)
        assert torch.isfinite(lse).all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("e,step", [(25, 8), (26, 8), (27, 16), (12, 16)])
@pytest.mark.parametrize("nq", [1, 12, 40])
def test_attention_maxima_sixteen_above_the_reference(nq, e, step, kind):
    """Logits (in powers of two) that are whole numbers at 2^e and rise by `step` with every fourth chunk of 32
    keys, so that a warp meets a maximum of 16 above its reference, where fp32's spacing is 4 to 16.  All of it is exact in
    fp32 but the last steps, so the tolerance takes no error of the logits."""
    rng = np.random.default_rng(15)
    page, d, n = 32, 64, 64
    c, r = pair(n, 1, d, 1, n, page, kind)
    fill(c, r, rng, [n * page])
    c.k.view(torch.int8).zero_()
    c.k.view(torch.int8)[..., 0] = 1 if kind == "int8" else 0x38    # 1
    r.k[:] = c.k.view(torch.uint8).cpu().numpy()
    r.k_scale[r.table[0, :n], 0] = np.float32(2.0 ** e + 1024 + step * (np.arange(n) // 4))
    c.k_scale.copy_(torch.from_numpy(r.k_scale))
    c.v_scale.fill_(1.0)
    r.v_scale[:] = 1.0
    q = torch.zeros((1, 1, nq, d), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    ln2 = float(np.float32(np.log(2.0)))  # sm_scale log2 e is 1 in fp32
    o, lse = sa.kv_attention(q.cuda(), c, causal=False, sm_scale=ln2)
    torch.cuda.synchronize()
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    want = list(r.attention(q.double().numpy(), False, sm_scale=ln2))
    want[4] = np.zeros_like(want[4])
    compare(o, lse, want, n * page, d)


@pytest.mark.parametrize("e", [8, 22, 34, 60])
@pytest.mark.parametrize("nq", [1, 40])
def test_attention_far_keys_before_near_ones(nq, e):
    """The first pages' logits lie at -2^(e + 3): the near keys behind them get their weights as if the
    far ones were not there."""
    rng = np.random.default_rng(e)
    far, n, d = 3, 570, 128
    c, r = pair(12, 1, d, 1, 10, 64, "int8")
    k = rng.standard_normal((1, 1, n, d)).astype(np.float32)
    k[:, :, :far * 64] = -np.abs(k[:, :, :far * 64])
    k = torch.from_numpy(k).to(torch.bfloat16)
    v, vf = bf16(rng, (1, 1, n, d))
    pos = sa.kv_extend(c, dev([n]))
    rpos, _ = r.extend([n])
    sa.kv_append(c, k.cuda(), v, pos, dev([n]))
    r.append(k.float().numpy(), vf, rpos, [n])
    same_state(c, r)
    q = torch.from_numpy(np.abs(rng.standard_normal((1, 2, nq, d))).astype(np.float32)).to(torch.bfloat16)
    qf = q.double().numpy()
    c.k_scale[:far] *= 2.0 ** e
    r.k_scale[:far] = 0.0
    near = r.attention(qf)[4]                 # max sum |q k| of the keys that count
    r.k_scale[:far] = c.k_scale[:far].cpu().numpy() * np.float32(2.0 ** (8 - e))   # e^-1000 is 0 as well
    o, lse, pv, av, mag, rows = r.attention(qf)
    assert mag.min() > 1000.0
    got = sa.kv_attention(q.cuda(), c)
    torch.cuda.synchronize()
    assert sa.get_status(c.status) == sa.SAGE_OK
    compare(*got, (o, lse, pv, av, near, rows), n, d)


@pytest.mark.parametrize("g,nq", [(1, 33), (4, 9), (8, 12), (1, 128)])
@pytest.mark.parametrize("page,d,kind", [(16, 64, "e4m3"), (64, 128, "int8"), (128, 128, "e4m3")])
def test_attention_one_row_tile(page, d, kind, g, nq):
    """33 to 128 query rows of a shared head: their key tiles are taken in turns.  Lengths of nothing, one, odd
    and even numbers of 128-key tiles, and one that is cut over many CTAs."""
    rng = np.random.default_rng(page + g + nq)
    lengths = [0, 1, 127, 128, 129, 256, 257, 385, 4501]
    c, r = pair(6000 // page + 40, 2, d, len(lengths), 4608 // page + 1, page, kind)
    fill(c, r, rng, lengths)
    check_attention(c, r, rng, 2 * g, nq, True, None, [nq, 1, nq, 0, nq - 1, nq, nq, nq // 2, nq])
    check_attention(c, r, rng, 2 * g, nq, False, [8, 4])


@pytest.mark.parametrize("d,kind", [(64, "int8"), (128, "e4m3")])
def test_attention_many_tiles_of_queries(d, kind):
    """Several 256-row units of each batch row, among rows with few or no queries, over short sequences."""
    rng = np.random.default_rng(d)
    c, r = pair(40, 2, d, 4, 10, 64, kind)
    fill(c, r, rng, [333, 0, 129, 64])
    check_attention(c, r, rng, 6, 600, True, [0, 2, 1, 3, 0], [600, 1, 599, 0, 86])
    check_attention(c, r, rng, 6, 600, False, [3, 2], [300, 600])


@pytest.mark.parametrize("nq", [1, 3, 40, 80])
def test_attention_queries_that_are_not_finite(nq):
    """A query of NaN or with an infinite element gives NaN in its own row, and nothing else changes."""
    rng = np.random.default_rng(21)
    c, r = pair(200, 2, 128, 3, 110, 64, "int8")
    fill(c, r, rng, [300, 77, 7000])
    q, _ = bf16(rng, (3, 4, nq, 128))
    o, lse = sa.kv_attention(q, c, causal=False)
    bad = torch.zeros((3, 4, nq), dtype=torch.bool, device="cuda")
    q2 = q.clone()
    for b, h in ((0, 1), (2, 3)):
        q2[b, h, 0] = float("nan")
        bad[b, h, 0] = True
    q2[1, 2, nq - 1, 5] = float("inf")
    bad[1, 2, nq - 1] = True
    o2, lse2 = sa.kv_attention(q2, c, causal=False)
    assert torch.isnan(o2[bad]).all() and torch.isnan(lse2[bad]).all()
    assert torch.equal(o2[~bad], o[~bad]) and torch.equal(lse2[~bad], lse[~bad])
    assert sa.get_status(c.status) == sa.SAGE_OK


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_bad_numbers_are_reported(nq):
    """A length past the table, a slot and a page out of range: reported, nothing read out of range,
    the other rows as ever."""
    rng = np.random.default_rng(9)
    c, r = pair(40, 1, 64, 4, 4, 16, "int8")
    fill(c, r, rng, [40, 20, 33, 10])
    q, qf = bf16(rng, (4, 2, nq, 64))
    want = r.attention(qf.astype(np.float64))

    def same(o, lse, rows):
        compare(o[rows], lse[rows], [x[rows] for x in want], 40, 64)

    same(*sa.kv_attention(q, c), [0, 1, 2, 3])
    assert sa.get_status(c.status) == sa.SAGE_OK
    c.lengths[0] = 65
    c.table[2, 1] = 40
    o, lse = sa.kv_attention(q, c)
    assert sa.get_status(c.status) == sa.SAGE_ERR_INVALID_ARG
    same(o, lse, [1, 3])
    assert not o[0].any() and (lse[0] == -np.inf).all()
    c.lengths[0] = -1
    sa.kv_attention(q, c)
    assert sa.get_status(c.status) == sa.SAGE_ERR_INVALID_ARG
    c.lengths[0] = 40
    o, lse = sa.kv_attention(q, c, slots=dev([1, 4, -1, 3]))
    assert sa.get_status(c.status) == sa.SAGE_ERR_INVALID_ARG
    same(o, lse, [3])
    assert not o[1].any() and not o[2].any()


@pytest.mark.parametrize("bad", [-1, 60, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("page,d,kind", [(16, 64, "int8"), (64, 128, "e4m3"), (128, 128, "int8"), (32, 64, "e4m3")])
@pytest.mark.parametrize("nq", [1, 16, 40, 100, 300])
def test_attention_leaves_out_a_page_out_of_range(nq, page, d, kind, bad):
    """A page number out of range inside a sequence: reported, its keys left out and nothing put in their place,
    as if the sequence did not have them.  The last page (partly filled) likewise."""
    rng = np.random.default_rng(page + nq)
    c, r = pair(60, 2, d, 3, 12, page, kind)
    fill(c, r, rng, [8 * page + 5, 40, 9 * page])
    q, qf = bf16(rng, (3, 4, nq, d))
    qf = qf.astype(np.float64)
    n = 9 * page
    for at, gone, causals in ((8, 5, (False,)), (1, page, (True, False) if nq + 2 * page <= n else (False,))):
        kept, table = int(c.table[0, at]), r.table[0].copy()
        c.table[0, at] = bad
        r.table[0, at:-1] = r.table[0, at + 1:].copy()
        r.lengths[0] -= gone
        for causal in causals:
            o, lse = sa.kv_attention(q, c, causal=causal)
            assert sa.get_status(c.status) == sa.SAGE_ERR_INVALID_ARG
            compare(o, lse, r.attention(qf, causal), n, d)
        c.table[0, at] = kept
        r.table[0], r.lengths[0] = table, r.lengths[0] + gone


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,hkv,g,nq", [(3, 2, 1, 1), (7, 2, 8, 3), (40, 2, 4, 1), (2, 3, 2, 70), (40, 2, 2, 200)])
def test_join_leaves_units_whose_parts_were_not_written(B, hkv, g, nq, d):
    """What a wait that ran out leaves: parts of units that nobody wrote, here numbers out of range in every way.  Their
    rows stay as they were, and the units beside them are joined."""
    rng = np.random.default_rng(B + nq)
    c = sa.kv_cache(1, hkv, d, B, 1)
    rows = g * nq
    R = 8 if rows <= 8 else 16 if rows <= 32 else 256
    tiles = -(-rows // R)
    units, most = B * tiles * hkv, 160 if R == 256 else 512
    ws = sa.alloc_kv_ws(c, B, hkv * g, nq)
    at, stride = (units * 8 + 255) // 256 * 256 // 4, R * (d + 2)
    assert ws.numel() == 4 * (at + 2 * most * stride)
    ws.view(torch.float32).fill_(float("nan"))
    bad = [(-1, 1), (0, most), (3, 2 ** 31 - 1), (-2 ** 31, 2 ** 31 - 1), (-2, -1), (5, 3), (2 ** 31 - 1, -2 ** 31), (7, 7),
           (most, most + 1), (-2 ** 31, 5), (most - 1, most)]
    info = np.array([bad[i % len(bad)] for i in range(units)], np.int32)
    # two units are as a call leaves them: one in parts 2 to 4, one in the workspace's last two
    good = {units // 2: (2, 4), units - 1: (most - 2, most - 1)}
    parts = torch.zeros((2 * most, R * (d + 2)))
    sums, m, l = {}, {}, {}
    for u, (a, b) in good.items():
        info[u] = a, b
        for k in range(a, b + 1):
            x = torch.from_numpy(rng.standard_normal((R, d)).astype(np.float32))
            top, low = torch.from_numpy(rng.integers(-3, 4, R).astype(np.float32)), torch.from_numpy(rng.uniform(0.5, 2, R).astype(np.float32))
            parts[2 * k + (k == a)] = torch.cat((x.flatten(), top, low))
            sums[u, k], m[u, k], l[u, k] = x.double(), top.double(), low.double()
    flat = ws.view(torch.float32)
    for u, (a, b) in good.items():
        for k in range(a, b + 1):
            i = 2 * k + (k == a)
            flat[at + i * stride:at + (i + 1) * stride] = parts[i].cuda()
    ws.view(torch.int32)[:2 * units] = torch.from_numpy(info.reshape(-1)).cuda()
    o = torch.full((B, hkv * g, nq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, hkv * g, nq), 7.0, device="cuda")
    rc = sa.sage_attn_selftest_kv_join(c._ref, o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.nbytes, B, hkv * g, nq,
                                       torch.cuda.current_stream().cuda_stream)
    assert rc == sa.SAGE_OK
    torch.cuda.synchronize()
    go, gl = o.double().cpu(), lse.double().cpu()
    want_o, want_l = torch.full_like(go, 7.0), torch.full_like(gl, 7.0)
    for u, (a, b) in good.items():
        bt, hk = divmod(u, hkv)
        bi, tile = divmod(bt, tiles)
        w = [2.0 ** m[u, k] for k in range(a, b + 1)]
        total = sum(f * l[u, k] for f, k in zip(w, range(a, b + 1)))
        joined = sum(f[:, None] * sums[u, k] for f, k in zip(w, range(a, b + 1))) / total[:, None]
        for x in range(R):
            row = tile * R + x
            if row < rows:
                want_o[bi, hk * g + row % g, row // g] = joined[x]
                want_l[bi, hk * g + row % g, row // g] = torch.log(total[x])
    # Each of up to three terms and the row sum is off by ex2's 2^-22 and a few roundings of 2^-24, O by both: 2^-20
    # of sum w |x| / total <= max |x| / 0.5; then bf16's half step.
    tol = 2.0 ** -8 * want_o.abs() + 2.0 ** -19 * (1 + 2.0 ** -8) * max(float(x.abs().max()) for x in sums.values())
    assert ((go - want_o).abs() <= tol).all() and ((gl - want_l).abs() <= 2.0 ** -19 * (1 + want_l.abs())).all()


@pytest.mark.parametrize("nq", [3, 40])
def test_attention_query_counts_out_of_range(nq):
    """q_len below 0 counts as 0, above Nq as Nq."""
    rng = np.random.default_rng(22)
    c, r = pair(30, 2, 128, 3, 8, 32, "int8")
    fill(c, r, rng, [50, 7, 120])
    q, qf = bf16(rng, (3, 4, nq, 128))
    for given, counts in (([-5, nq + 9, 2], [0, nq, 2]), ([2 ** 31 - 1, -2 ** 31, nq], [nq, 0, nq])):
        o, lse = torch.full_like(q, 7.0), torch.full((3, 4, nq), 7.0, device="cuda")
        sa.kv_attention(q, c, q_len=dev(given), o=o, lse=lse)
        torch.cuda.synchronize()
        assert sa.get_status(c.status) == sa.SAGE_OK
        compare(o, lse, r.attention(qf.astype(np.float64), True, None, counts), 120, 128)


@pytest.mark.parametrize("d,g,nq", [(64, 1, 1), (128, 4, 4), (128, 1, 40)])
def test_attention_most_batch_rows(d, g, nq):
    """4096 rows over 40 slots, each kernel."""
    rng = np.random.default_rng(23)
    c, r = pair(64, 1, d, 40, 4, 16, "int8")
    fill(c, r, rng, 1 + np.arange(40) % 33)
    slots = np.arange(4096) % 40
    q, qf = bf16(rng, (4096, g, nq, d))
    o, lse = sa.kv_attention(q, c, slots=dev(slots))
    torch.cuda.synchronize()
    assert sa.get_status(c.status) == sa.SAGE_OK
    some = list(range(40)) + [2047, 3333, 4095]
    compare(o[some], lse[some], r.attention(qf[some].astype(np.float64), True, slots[some]), 33, d)


def test_attentions_at_once_over_one_cache():
    """Calls on two streams, each with its own workspace, read one cache at the same time."""
    rng = np.random.default_rng(24)
    c, r = pair(300, 2, 128, 3, 150, 32, "e4m3")
    fill(c, r, rng, [50, 4500, 120])
    many, manyf = bf16(rng, (3, 4, 20, 128))
    one, onef = bf16(rng, (3, 4, 1, 128))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        x, y, z = sa.kv_attention(many, c, stream=a), sa.kv_attention(one, c, stream=b), sa.kv_attention(many, c, stream=b)
    torch.cuda.synchronize()
    assert sa.get_status(c.status) == sa.SAGE_OK
    compare(*x, r.attention(manyf.astype(np.float64)), 4500, 128)
    compare(*y, r.attention(onef.astype(np.float64)), 4500, 128)
    assert torch.equal(x[0], z[0]) and torch.equal(x[1], z[1])


def test_attention_offsets_past_32_bits():
    """A pool of more than 2^32 codes, the sequence in its last pages."""
    rng = np.random.default_rng(10)
    n_pages, hkv, d, page = 33000, 8, 128, 128
    kind = "e4m3"
    c = sa.KVCache(*[torch.empty((n_pages, hkv, page, d), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)],
                   *[torch.empty((n_pages, hkv), device="cuda") for _ in range(2)],
                   torch.zeros((1, 8), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                   torch.ones(n_pages, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert n_pages * hkv * page * d > 2 ** 32
    c.refs[-8:] = 0
    r = kv_ref.Cache(8, hkv, d, 1, 8, page, kind)
    n = 700
    pos = sa.kv_extend(c, dev([n]))
    rpos, _ = r.extend([n])
    assert np.array_equal(c.table[0, :6].cpu().numpy() - (n_pages - 8), r.table[0, :6])
    k, kf = bf16(rng, (1, hkv, n, d))
    v, vf = bf16(rng, (1, hkv, n, d))
    sa.kv_append(c, k, v, pos, dev([n]))
    r.append(kf, vf, rpos, [n])
    torch.cuda.synchronize()
    assert np.array_equal(c.k[-8:-2].view(torch.uint8).cpu().numpy(), r.k[:6])
    check_attention(c, r, rng, 16, 1)
    check_attention(c, r, rng, 16, 20)


# ------------------------------------------------------------------------------ pages

@pytest.mark.parametrize("seed", range(4))
def test_pages_random_walk(seed):
    """Forks, extensions (shared last pages copied, pools that run out), truncations and compactions in a
    random order, the state compared bit for bit after each."""
    rng = np.random.default_rng(seed)
    S, M, page = 9, 6, 16
    c, r = pair(24, 2, 64, S, M, page, "int8", poison=False)
    for step in range(30):
        what = rng.integers(0, 4)
        expect = {sa.SAGE_OK}
        if what == 0:
            src = np.where(rng.random(S) < 0.4, rng.integers(-1, S, S), -1)
            if any(f >= 0 and (src[f] >= 0 or r.lengths[s]) for s, f in enumerate(src)):
                expect = {sa.SAGE_ERR_INVALID_ARG}
            sa.kv_fork(c, dev(src))
            r.fork(src)
        elif what == 1:
            n = np.where(rng.random(S) < 0.6, rng.integers(0, 2 * page, S), 0)
            pos, cow = torch.empty(S, dtype=torch.int32, device="cuda"), torch.empty(S, dtype=torch.int32, device="cuda")
            sa.kv_extend(c, dev(n), pos=pos, cow=cow)
            rpos, rcow = r.extend(n)
            assert np.array_equal(pos.cpu().numpy(), rpos) and np.array_equal(cow.cpu().numpy(), rcow)
            if (rpos < 0).any():
                expect = {sa.SAGE_ERR_NO_PAGES, sa.SAGE_ERR_INVALID_ARG}
            k, kf = bf16(rng, (S, 2, max(1, n.max()), 64))
            sa.kv_append(c, k, k, pos, dev(n))
            r.append(kf, kf, rpos, n)
        elif what == 2:
            keep = np.where(rng.random(S) < 0.5, rng.integers(0, M * page, S), -1)
            sa.kv_truncate(c, dev(keep))
            r.truncate(keep)
        else:
            c2, r2 = pair(24 + step % 3, 2, 64, S, M, page, "int8", poison=False)
            sa.kv_compact(c, c2)
            if r.compact(r2):
                assert sa.get_status(c.status) == sa.SAGE_OK
                c, r = c2, r2
            else:
                same_state(c2, r2)
                expect = {sa.SAGE_ERR_NO_PAGES}
        same_state(c, r)
        assert sa.get_status(c.status) in expect
        live = np.zeros(len(r.refs), np.int32)
        for s in range(S):
            live += np.bincount(r.table[s, :r.pages(int(r.lengths[s]))], minlength=len(live)).astype(np.int32)
        assert np.array_equal(live, r.refs)


def test_extend_many_slots_and_pages():
    """More slots than the kernel has threads, more pages than one step of its scan looks at; an
    exact fit, then a pool without a page left."""
    rng = np.random.default_rng(2)
    S, N = 2500, 40000
    c = sa.kv_cache(N, 1, 64, S, 30, page=16)
    r = kv_ref.Cache(N, 1, 64, S, 30, 16, "int8")
    taken = rng.random(N) < 0.3
    c.refs.copy_(dev(taken))
    r.refs[:] = taken
    n = rng.integers(0, 150, S)
    assert np.array_equal(sa.kv_extend(c, dev(n)).cpu().numpy(), r.extend(n)[0])
    same_state(c, r)
    left = int((r.refs == 0).sum())
    room = 30 * 16 - r.lengths
    n = np.zeros(S, np.int64)
    for s in range(S):  # whole pages until exactly none is left
        give = min(left, room[s] // 16)
        n[s] = give * 16
        left -= give
    assert left == 0
    pos = sa.kv_extend(c, dev(n))
    assert np.array_equal(pos.cpu().numpy(), r.extend(n)[0]) and (pos >= 0).all() and sa.get_status(c.status) == sa.SAGE_OK
    same_state(c, r)
    assert (r.refs > 0).all()
    n = np.ones(S, np.int64)
    assert np.array_equal(sa.kv_extend(c, dev(n)).cpu().numpy(), r.extend(n)[0])
    same_state(c, r)
    # some slots ask for more than their table holds: of two errors the word keeps that one
    assert (r.lengths == 480).any() and sa.get_status(c.status) == sa.SAGE_ERR_INVALID_ARG
    n = (r.lengths < 480).astype(np.int64)
    assert np.array_equal(sa.kv_extend(c, dev(n)).cpu().numpy(), r.extend(n)[0])
    same_state(c, r)
    assert sa.get_status(c.status) == sa.SAGE_ERR_NO_PAGES


def test_extend_asks_for_more_than_there_can_be():
    """Needs whose sum passes 32 bits: nothing is served behind the first one that does not fit."""
    S = 100  # (100 slots of 2^25 pages: a table of 13 GB)
    c = sa.kv_cache(50, 1, 64, S, 2 ** 25, page=16)
    r = kv_ref.Cache(50, 1, 64, S, 4, 16, "int8")
    n = np.full(S, 2 ** 29 - 4096)
    n[:3] = [17, 0, 40]
    pos = sa.kv_extend(c, dev(n)).cpu().numpy()
    assert pos[:3].tolist() == [0, 0, 0] and (pos[3:] == -1).all()
    r.extend([17, 0, 40] + [0] * (S - 3))
    assert np.array_equal(c.lengths.cpu().numpy(), r.lengths) and np.array_equal(c.refs.cpu().numpy(), r.refs)
    assert sa.get_status(c.status) == sa.SAGE_ERR_NO_PAGES


def test_compact_too_small_and_refusals():
    rng = np.random.default_rng(4)
    c, r = pair(12, 1, 64, 3, 6, 16, "e4m3", poison=False)
    fill(c, r, rng, [40, 33, 7])
    to, rt = pair(6, 1, 64, 3, 6, 16, "e4m3", poison=False)
    sa.kv_compact(c, to)
    same_state(to, rt)  # seven live pages do not fit in six: left alone
    assert sa.get_status(c.status) == sa.SAGE_ERR_NO_PAGES
    to, rt = pair(7, 1, 64, 3, 6, 16, "e4m3", poison=False)
    to.refs.fill_(3)
    sa.kv_compact(c, to)
    r.compact(rt)
    same_state(to, rt)
    with pytest.raises(sa.SageError):
        sa.kv_compact(c, c)
    with pytest.raises(ValueError):
        sa.kv_extend(c, dev([1, 2]))
    with pytest.raises(ValueError):
        sa.kv_attention(torch.zeros((1, 1, 1, 64), device="cuda"), c)  # fp32 queries
    with pytest.raises(ValueError):
        sa.kv_attention(torch.zeros((4, 1, 1, 64), dtype=torch.bfloat16, device="cuda"), c)  # rows without slots
    with pytest.raises(ValueError):
        q = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
        sa.kv_attention(q, c, slots=dev([0]))


@pytest.mark.parametrize("bad", ["free", -1, 12, -2 ** 31])
def test_compact_reports_listed_pages_that_are_not_live(bad):
    rng = np.random.default_rng(16)
    c, r = pair(12, 1, 64, 2, 6, 16, "int8", poison=False)
    fill(c, r, rng, [40, 20])
    to, _ = pair(12, 1, 64, 2, 6, 16, "int8", poison=False)
    if bad == "free":
        c.refs[int(r.table[0, 1])] = 0
    else:
        c.table[0, 1] = bad
    sa.kv_compact(c, to)
    assert sa.get_status(c.status) == sa.SAGE_ERR_INVALID_ARG
    assert sa.get_status(to.status) == sa.SAGE_OK
    assert int(to.table[0, 1]) == -1 and (to.table[0, [0, 2]] >= 0).all() and (to.table[1, :2] >= 0).all()
    q, _ = bf16(rng, (2, 1, 1, 64))
    sa.kv_attention(q, to)                # and what reads it says so too
    assert sa.get_status(to.status) == sa.SAGE_ERR_INVALID_ARG


def test_workspaces_with_gaps_are_refused():
    """A strided view has the bytes asked for, but not one behind the other."""
    rng = np.random.default_rng(20)
    c, r = pair(8, 1, 64, 2, 4, 16, "int8", poison=False)
    fill(c, r, rng, [20, 9])
    to = sa.kv_cache(8, 1, 64, 2, 4, page=16)
    q, _ = bf16(rng, (2, 1, 1, 64))
    for ws, call in ((sa.alloc_kv_ws(c, 2, 1, 1), lambda w: sa.kv_attention(q, c, ws=w)),
                     (sa.alloc_kv_compact_ws(c), lambda w: sa.kv_compact(c, to, ws=w))):
        big = torch.full((2 * ws.numel(),), 77, dtype=torch.uint8, device="cuda")
        with pytest.raises(ValueError, match="contiguous"):
            call(big[::2])
        torch.cuda.synchronize()
        assert (big == 77).all()
        call(big[:ws.numel()])
        with pytest.raises(sa.SageError):
            call(ws[:-1])
        with pytest.raises(ValueError):
            call(ws.cpu())
    assert sa.get_status(c.status) == sa.SAGE_OK


# ------------------------------------------------------------------------------ together

def test_serving_run_in_graphs_and_streams():
    """As a server uses them: prompts, a fork into samples, a decoding step captured once and replayed
    while lengths, pages and inputs change, on a stream of its own; a second captured graph (another
    batch) shares the workspace.  Every step against the reference."""
    rng = np.random.default_rng(6)
    S, H, hkv, d = 6, 8, 2, 128
    c, r = pair(64, hkv, d, S, 12, 16, "int8", poison=False)
    fill(c, r, rng, [50, 33, 0, 0, 0, 0])
    src = [-1, -1, 0, 0, 1, 1]
    sa.kv_fork(c, dev(src))
    r.fork(src)
    n = dev(np.ones(S))
    k, v = (torch.zeros((S, hkv, 1, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((S, H, 1, d), dtype=torch.bfloat16, device="cuda")
    pos, cow = torch.empty_like(n), torch.empty_like(n)
    o, lse = torch.empty_like(q), torch.empty((S, H, 1), device="cuda")
    ws = sa.alloc_kv_ws(c, S, H, 1)
    q2 = torch.zeros((2, H, 1, d), dtype=torch.bfloat16, device="cuda")
    o2, lse2 = torch.empty_like(q2), torch.empty((2, H, 1), device="cuda")
    slots2 = dev([5, 0])
    assert sa.alloc_kv_ws(c, 2, H, 1).numel() <= ws.numel()

    def step():
        sa.kv_extend(c, n, pos=pos, cow=cow)
        sa.kv_append(c, k, v, pos, n)
        sa.kv_attention(q, c, o=o, lse=lse, ws=ws)

    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    saved = [t.clone() for t in (c.lengths, c.refs, c.table, c.k.view(torch.int8), c.v.view(torch.int8), c.k_scale, c.v_scale)]
    with torch.cuda.stream(stream):
        step()  # (and back)
        for t, x in zip((c.lengths, c.refs, c.table, c.k.view(torch.int8), c.v.view(torch.int8), c.k_scale, c.v_scale), saved):
            t.copy_(x)
        stream.synchronize()
        graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        with torch.cuda.graph(graph2, stream=stream):
            sa.kv_attention(q2, c, slots=slots2, o=o2, lse=lse2, ws=ws)
    for i in range(20):
        kb, kf = bf16(rng, (S, hkv, 1, d))
        vb, vf = bf16(rng, (S, hkv, 1, d))
        qb, qf = bf16(rng, (S, H, 1, d))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            k.copy_(kb), v.copy_(vb), q.copy_(qb), q2.copy_(qb[[5, 0]])
            graph.replay()
            graph2.replay()
        torch.cuda.synchronize()
        one = np.ones(S, np.int64)
        rpos, _ = r.extend(one)
        r.append(kf, vf, rpos, one)
        same_state(c, r)
        want = r.attention(qf.astype(np.float64))
        compare(o, lse, want, 80, d)
        compare(o2, lse2, [x[[5, 0]] for x in want], 80, d)
    assert sa.get_status(c.status) == sa.SAGE_OK
    # the same call twice gives the same bits
    a, b = (sa.kv_attention(q, c) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    keep = [0, -1, 10, 0, 0, 60]
    sa.kv_truncate(c, dev(keep))
    r.truncate(keep)
    c2, r2 = pair(20, hkv, d, S, 12, 16, "int8", poison=False)
    sa.kv_compact(c, c2)
    r.compact(r2)
    same_state(c2, r2)
    check_attention(c2, r2, rng, H, 5, q_len=[5, 3, 1, 5, 5, 5])


def test_helpers_on_a_given_stream(monkeypatch):
    """What a helper allocates for a call on another stream is not given away while that stream still
    has to use it."""
    from bit_trainable_attention_sagebwd_gb300 import kvcache
    rng = np.random.default_rng(2)
    c, r = pair(20, 2, 64, 3, 8, 32, "int8")
    k, kf = bf16(rng, (3, 2, 50, 64))
    q, qf = bf16(rng, (3, 4, 1, 64))
    n = dev([50, 7, 0])
    held = []

    def kept(alloc):
        def call(*args):
            t = alloc(*args)
            held.append((t.data_ptr(), t.nbytes))
            return t
        return call
    monkeypatch.setattr(kvcache, "alloc_kv_ws", kept(kvcache.alloc_kv_ws))
    monkeypatch.setattr(kvcache, "alloc_kv_compact_ws", kept(kvcache.alloc_kv_compact_ws))
    to = sa.kv_cache(30, 2, 64, 3, 8, page=32)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(200_000_000)        # about 0.1 s
    pos = sa.kv_extend(c, n, stream=stream)
    sa.kv_append(c, k, k, pos, n, stream=stream)
    o, lse = sa.kv_attention(q, c, stream=stream)
    sa.kv_compact(c, to, stream=stream)
    assert not stream.query()
    assert len(held) == 2
    for ptr, size in held:
        later = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert all(t.data_ptr() != ptr for t in later)
    stream.synchronize()
    rpos, _ = r.extend([50, 7, 0])
    r.append(kf, kf, rpos, [50, 7, 0])
    same_state(c, r)
    assert np.array_equal(pos.cpu().numpy(), rpos)
    compare(o, lse, r.attention(qf.astype(np.float64)), 50, 64)
    assert torch.equal(to.lengths, c.lengths)


def test_helpers_on_a_given_stream_take_memory_of_that_stream():
    """What a helper allocates for a call on another stream is not memory that the current stream, which the call
    does not wait for, still has work on; and what it returned is not given away under the current stream's work."""
    rng = np.random.default_rng(18)
    c, r = pair(20, 2, 64, 3, 8, 32, "int8")
    fill(c, r, rng, [50, 7, 120])
    q, qf = bf16(rng, (3, 4, 1, 64))
    q2, _ = bf16(rng, (3, 4, 1, 64))
    want = r.attention(qf.astype(np.float64))
    n = dev([3, 0, 40])
    rpos, _ = r.extend([3, 0, 40])
    to = sa.kv_cache(30, 2, 64, 3, 8, page=32)
    sizes = [sa.alloc_kv_ws(c, 3, 4, 1).nbytes, q.nbytes, 3 * 4 * 4, n.nbytes, n.nbytes, sa.alloc_kv_compact_ws(c).nbytes]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()              # what is freed below is what an allocation on the current stream gets
    freed = [torch.empty(size, dtype=torch.uint8, device="cuda") for size in sizes]
    torch.cuda._sleep(200_000_000)        # about 0.1 s
    for t in freed:
        t.fill_(255)                      # NaN, -1: while or after the calls below work
    places = {t.data_ptr() for t in freed}
    t = freed = None
    o, lse = sa.kv_attention(q, c, stream=stream)
    pos = sa.kv_extend(c, n, stream=stream)
    sa.kv_compact(c, to, stream=stream)
    torch.cuda.synchronize()
    assert places.isdisjoint({o.data_ptr(), lse.data_ptr(), pos.data_ptr()})
    compare(o, lse, want, 120, 64)
    assert np.array_equal(pos.cpu().numpy(), rpos) and torch.equal(to.lengths, c.lengths)
    assert sa.get_status(c.status) == sa.SAGE_OK
    kept, place = o.clone(), o.data_ptr()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    later = o.clone()                     # the current stream still has to read o
    o = None
    o2, _ = sa.kv_attention(q2, c, stream=stream)
    assert o2.data_ptr() != place or torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert torch.equal(later, kept) and not torch.equal(o2, kept)


def test_calls_of_two_threads():
    """Two host threads, each with its own stream, caches and workspaces, whose calls differ in what they take of an
    SM's shared memory (batch rows of an attention, slots of an extend)."""
    rng = np.random.default_rng(19)
    d, many = 128, 700
    jobs = []
    for rows, slots in ((2, 5200), (many, 8192)):
        c, r = pair(many + 8, 1, d, many, 2, 16, "int8")
        fill(c, r, rng, 1 + np.arange(many) % 5)
        q, qf = bf16(rng, (rows, 1, 1, d))
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            ws = sa.alloc_kv_ws(c, rows, 1, 1)
            o, lse = torch.empty_like(q), torch.empty((rows, 1, 1), device="cuda")
            big = sa.kv_cache(slots, 1, 64, slots, 1, page=16)
            n = torch.ones(slots, dtype=torch.int32, device="cuda")
            pos, cow = torch.empty_like(n), torch.empty_like(n)
        jobs.append((c, r, q, qf, stream, ws, o, lse, big, n, pos, cow))
    torch.cuda.synchronize()
    start, failed = threading.Barrier(2), []

    def work(c, r, q, qf, stream, ws, o, lse, big, n, pos, cow):
        try:
            start.wait()
            for i in range(300):
                sa.kv_attention(q, c, slots=slots_of[len(q)], o=o, lse=lse, ws=ws, stream=stream)
                if i < 16:
                    sa.kv_extend(big, n, pos=pos, cow=cow, stream=stream)
        except Exception as e:
            failed.append(e)

    slots_of = {len(j[2]): dev(np.arange(len(j[2]))) for j in jobs}
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for c, r, q, qf, stream, ws, o, lse, big, n, pos, cow in jobs:
        assert sa.get_status(c.status) == sa.SAGE_OK and sa.get_status(big.status) == sa.SAGE_OK
        compare(o, lse, r.attention(qf.astype(np.float64), slots=list(range(len(q)))), 5, d)
        assert (big.lengths == 16).all() and (big.refs == 1).all()


def test_prompt_in_chunks_equals_prompt_at_once():
    """A prompt attended over in chunks against the same prompt in one call (the same cache)."""
    rng = np.random.default_rng(7)
    c, r = pair(20, 2, 128, 1, 20, 64, "e4m3")
    fill(c, r, rng, [300])
    q, o, lse = check_attention(c, r, rng, 4, 300)
    c.lengths.fill_(0)
    at = 0
    for n in (64, 1, 100, 135):
        c.lengths.add_(n)
        r.lengths[0] = at + n
        part = q[:, :, at:at + n].contiguous()
        po, pl = torch.full_like(part, 7.0), torch.full((1, 4, n), 7.0, device="cuda")
        sa.kv_attention(part, c, o=po, lse=pl)
        torch.cuda.synchronize()
        compare(po, pl, r.attention(part.double().cpu().numpy()), 300, 128)
        at += n
