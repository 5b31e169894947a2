"""Calls of the packed attention and the rotary positions as programs make them: together, with the key/value cache, on
several streams, with strides past 32 bits, with sequences that the workspace's line of work cuts anywhere; on the GPU."""
import random

import pytest
import torch

import bit_trainable_attention_sagebwd_gb300 as sa
import packed_ref as ref
from test_gpu_packed import backward_checked, forward_checked
from test_gpu_rotary import check, ints, table, turned, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def fp32_default():
    """torch's default type as it is for a user: another module of the run may have changed it."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


def places(lens):
    return torch.cat([torch.arange(n) for n in lens]).cuda()


# ------------------------------------------------------------------- together

@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (64, 32, True)])
def test_a_training_step(D, rot, interleaved):
    """Turn, attend, and both backwards, all but the projections' own arithmetic from views of one fused projection;
    each result against the formulas at what the step before it gave."""
    lens, H, Hkv = [200, 1, 0, 333, 64], 6, 2
    T = sum(lens)
    t, freq, gain = table(rot, interleaved, scaling="ramp", factor=4.0, context=128)
    fused = values(T, H + 2 * Hkv, D)
    q, k, v = fused.split([H, Hkv, Hkv], 1)
    do = values(T, H, D, seed=1)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    pos = places(lens)
    want = [turned(x.transpose(0, 1), pos, freq, rot, interleaved, gain, False) for x in (q, k)]
    sa.rotary(t, q, k, cu_seqlens=cu, q_out=q, k_out=k)
    for x, w in zip((q, k), want):
        check(x.transpose(0, 1), w)
    forward_checked(q, k, v, cu, True)
    grads = torch.zeros_like(fused)
    dq, dk, dv = grads.split([H, Hkv, Hkv], 1)
    backward_checked(q, k, v, do, cu, True, dq=dq, dk=dk, dv=dv)
    want = [turned(x.transpose(0, 1), pos, freq, rot, interleaved, gain, True) for x in (dq, dk)]
    sa.rotary_backward(t, dq, dk, cu_seqlens=cu, q_out=dq, k_out=dk)
    for x, w in zip((dq, dk), want):
        check(x.transpose(0, 1), w)


def test_prompts_and_then_tokens():
    """Prompts of different lengths packed, their keys and values stored, and a further token of each: turned by the
    cache's own positions and attended with the cache."""
    lens, H, Hkv, D, page = [130, 47, 64], 4, 2, 128, 64
    S, T, N = len(lens), sum(lens), max(lens)
    t, _, _ = table(D, False, scaling="linear", factor=2.0)
    # every sequence with one token more than its prompt
    whole = [n + 1 for n in lens]
    cu1 = torch.tensor([0] + whole).cumsum(0).to(torch.int32).cuda()
    raw = values(T + S, H, D), values(T + S, Hkv, D, seed=1), values(T + S, Hkv, D, seed=2)
    prompt = torch.cat([torch.arange(b, b + n) for b, n in zip(cu1.tolist(), lens)]).cuda()
    token = (cu1[1:] - 1).long()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    q, k, v = (x[prompt] for x in raw)
    sa.rotary(t, q, k, cu_seqlens=cu, q_out=q, k_out=k)
    o, _ = forward_checked(q, k, v, cu, True)

    c = sa.kv_cache(16, Hkv, D, S, 4, page=page, kind="e4m3")
    n = ints(*lens)
    padded = []
    for x in (k, v):
        p = torch.zeros((S, Hkv, N, D), dtype=torch.bfloat16, device="cuda")
        for s, (b, m) in enumerate(zip(cu.tolist(), lens)):
            p[s, :, :m] = x[b:b + m].transpose(0, 1)
        padded.append(p)
    sa.kv_append(c, *padded, sa.kv_extend(c, n), n)
    # the tokens
    pos = sa.kv_extend(c, torch.ones_like(n))
    q1, k1, v1 = (x[token].unsqueeze(2).contiguous() for x in raw)
    q1, k1 = sa.rotary(t, q1, k1, start=pos)
    sa.kv_append(c, k1, v1, pos, torch.ones_like(n))
    o1, _ = sa.kv_attention(q1, c, slots=ints(0, 1, 2))
    assert sa.get_status(c.status) == sa.SAGE_OK
    # the same turn as in the whole sequence
    qw, kw = sa.rotary(t, raw[0], raw[1], cu_seqlens=cu1)
    assert torch.equal(qw[prompt], q) and torch.equal(kw[prompt], k)
    assert torch.equal(qw[token], q1[:, :, 0]) and torch.equal(kw[token], k1[:, :, 0])
    # the prompts' rows do not see the token; the token's do, through the cache's 8 bits
    ow, _ = sa.packed_forward(qw, kw, raw[2], cu1)
    assert ((ow[prompt].double() - o.double()).abs() <= 2.0 ** -7 * v.double().abs().max()).all()
    for s, m in enumerate(whole):
        ids = c.table[s, :-(-m // page)].long()
        for h in range(H):
            ks, vs = ((x[ids, h // 2].double() * y[ids, h // 2].double()[:, None, None]).reshape(-1, D)[:m]
                      for x, y in ((c.k, c.k_scale), (c.v, c.v_scale)))
            want = torch.softmax(q1[s, h].double() @ ks.T / D ** 0.5, -1) @ vs
            # rounding of P (2^-11) and O (2^-8) of the largest value
            assert (o1[s, h].double() - want).abs().max() <= 2.0 ** -7 * vs.abs().max()


# ------------------------------------------------------------------- work cut anywhere

@pytest.mark.parametrize("seed", range(8))
def test_lengths_at_random(seed):
    rng = random.Random(seed)
    D, G, Hkv, causal = rng.choice((64, 128)), rng.choice((1, 2, 3, 4, 5, 8, 12)), rng.choice((1, 2, 3)), rng.random() < 0.7
    most = rng.choice((20, 200, 900))
    lens = [rng.choice((0, 1, rng.randint(1, most), rng.randint(1, most))) for _ in range(rng.randint(1, 3000 // most))] + [1]
    q, k, v, do, cu = ref.inputs(lens, G * Hkv, Hkv, D, seed=seed, before=rng.randint(0, 9), behind=rng.randint(0, 200))
    forward_checked(q, k, v, cu, causal)
    backward_checked(q, k, v, do, cu, causal)


@pytest.mark.parametrize("lens,H,Hkv,D,causal", [([9001], 1, 1, 128, True), ([5000, 7], 3, 1, 64, False)], ids=str)
def test_one_long_sequence_over_many_ctas(lens, H, Hkv, D, causal):
    q, k, v, do, cu = ref.inputs(lens, H, Hkv, D)
    forward_checked(q, k, v, cu, causal)
    backward_checked(q, k, v, do, cu, causal)


def test_the_most_tokens_and_sequences():
    """2^24 tokens in 65536 sequences: those at the beginning, in the middle and at the end as if alone."""
    S, n, H, Hkv, D = 65536, 256, 2, 1, 64
    T = S * n
    g = torch.Generator("cuda").manual_seed(0)
    q, do = (torch.randn((T, H, D), device="cuda", generator=g, dtype=torch.bfloat16) for _ in range(2))
    k, v = (torch.randn((T, Hkv, D), device="cuda", generator=g, dtype=torch.bfloat16) for _ in range(2))
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda") * n
    cu[1:-1] += torch.randint(-100, 101, (S - 1,), device="cuda", generator=g, dtype=torch.int32)
    o, lse = sa.packed_forward(q, k, v, cu)
    ws = sa.alloc_packed_ws(T, S, H, Hkv, D, backward=True)
    grads = sa.packed_backward(q, k, v, o, lse, do, cu, ws=ws)
    assert sa.get_status(ws) == sa.SAGE_OK
    for s in (0, 127, 128, S // 2, S - 3):
        b, e = int(cu[s]), int(cu[s + 3])
        x = [y[b:e] for y in (q, k, v, do)]
        part = cu[s:s + 4] - b
        want = ref.forward(*x[:3], part, True, D ** -0.5)
        ref.check(o[b:e], want[0], want[2], f"O of {s}")
        ref.check(lse[:, b:e], want[1], want[3], f"LSE of {s}")
        want, tol = ref.backward(*x[:3], o[b:e], lse[:, b:e], x[3], part, True, D ** -0.5)
        for got, name in zip(grads, ("dq", "dk", "dv")):
            ref.check(got[b:e], want[name], tol[name], f"{name} of {s}")


@pytest.mark.parametrize("D,H,Hkv", [(128, 16, 16), (64, 16, 4)])
def test_gradients_of_many_documents(D, H, Hkv):
    """Many short units one behind the other on each SM, which nothing but the waits keeps apart."""
    lens = [101, 543, 119, 1298, 121, 194, 102, 1027, 727, 203, 336, 2048, 215, 107, 370, 329, 340, 251, 271, 190]
    q, k, v, do, cu = ref.inputs(lens, H, Hkv, D)
    o, lse, got = backward_checked(q, k, v, do, cu, True)
    for _ in range(10):
        for x, y in zip(got.values(), sa.packed_backward(q, k, v, o, lse, do, cu)):
            assert torch.equal(x, y)


# ------------------------------------------------------------------- workspaces

def test_a_workspace_full_of_anything():
    """Of the workspace only the header is read before it is written, and the header is left as it was."""
    q, k, v, do, cu = ref.inputs([2100, 5, 900], 4, 2, 128)
    want = sa.packed_forward(q, k, v, cu)
    grads = sa.packed_backward(q, k, v, *want, do, cu)
    ws = sa.alloc_packed_ws(3005, 3, 4, 2, 128, backward=True)
    for _ in range(3):
        ws[4096:] = 255
        got = sa.packed_forward(q, k, v, cu, ws=ws)
        assert not ws[:4096].any()
        ws[4096:] = 255
        back = sa.packed_backward(q, k, v, *want, do, cu, ws=ws)
        assert not ws[:4096].any()
        for x, y in zip((*got, *back), (*want, *grads)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("lens", [[0], [0, 0, 0]], ids=str)
def test_no_tokens_at_all(lens):
    q, k, v, do, _ = ref.inputs([70], 2, 1, 64)
    cu = torch.full((len(lens) + 1,), 9, dtype=torch.int32, device="cuda")
    ws = sa.alloc_packed_ws(70, len(lens), 2, 1, 64, backward=True)
    out = [torch.full_like(x, 7.0) for x in (q, q, k, k)]
    lse = torch.full((2, 70), 7.0, device="cuda")
    sa.packed_forward(q, k, v, cu, o=out[0], lse=lse, ws=ws)
    sa.packed_backward(q, k, v, out[0], lse, do, cu, dq=out[1], dk=out[2], dv=out[3], ws=ws)
    assert sa.get_status(ws) == sa.SAGE_OK
    assert all((x == 7).all() for x in (*out, lse))


@pytest.mark.parametrize("entries", [[0, 50, 110, 181], [-1, 50, 110, 180], [0, 2 ** 31 - 1, 110, 180], [0, 50, 40, 180],
                                     [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0]], ids=str)
def test_gradients_of_sequences_out_of_order_or_range_are_left_out(entries):
    q, k, v, do, cu = ref.inputs([180], 2, 1, 64)
    o, lse = sa.packed_forward(q, k, v, cu)
    ws = sa.alloc_packed_ws(180, 3, 2, 1, 64, backward=True)
    out = [torch.full_like(x, 7.0) for x in (q, k, k)]
    sa.packed_backward(q, k, v, o, lse, do, torch.tensor(entries, dtype=torch.int32, device="cuda"), dq=out[0], dk=out[1],
                       dv=out[2], ws=ws)
    assert sa.get_status(ws) == sa.SAGE_ERR_INVALID_ARG
    seen = torch.zeros(180, dtype=torch.bool)
    for b, e in zip(entries, entries[1:]):
        if 0 <= b <= e <= 180:
            seen[b:e] = True
    for x in out:
        assert (x[~seen.cuda()] == 7).all() and not x[seen.cuda()].isnan().any()


def test_sequences_over_one_another():
    """Entries that go up and down would be any amount of work; past twice the tokens none is done."""
    q, k, v, do, cu = ref.inputs([180], 2, 1, 64)
    o, lse = sa.packed_forward(q, k, v, cu)
    again = torch.tensor([0, 180] * 500 + [0], dtype=torch.int32, device="cuda")
    ws = sa.alloc_packed_ws(180, 1000, 2, 1, 64, backward=True)
    out = [torch.full_like(x, 7.0) for x in (q, q, k, k)]
    sa.packed_forward(q, k, v, again, o=out[0], ws=ws)
    assert sa.get_status(ws) == sa.SAGE_ERR_INVALID_ARG
    sa.packed_backward(q, k, v, o, lse, do, again, dq=out[1], dk=out[2], dv=out[3], ws=ws)
    assert sa.get_status(ws) == sa.SAGE_ERR_INVALID_ARG
    assert all((x == 7).all() for x in out)


def test_refusals():
    q, k, v, do, cu = ref.inputs([40, 30], 2, 1, 64)
    o, lse = sa.packed_forward(q, k, v, cu)
    ws = sa.alloc_packed_ws(70, 2, 2, 1, 64)
    for bad in (dict(o=q), dict(ws=ws[:-256]), dict(ws=ws[1:]), dict(o=o[:1].expand(70, 2, 64)), dict(sm_scale=float("nan"))):
        with pytest.raises(sa.SageError):
            sa.packed_forward(q, k, v, cu, **bad)
    for bad in (dict(o=o.float()), dict(o=o[1:]), dict(lse=lse.T), dict(ws=ws.cpu()), dict(ws=ws[::2]), dict(lse=lse.cpu()),
                dict(o=o.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            sa.packed_forward(q, k, v, cu, **bad)
    for bad in ((q, k, v, cu.long()), (q, k[:, :, :32], v, cu), (q, k, v.half(), cu), (q, k, v[1:], cu), (q, k, v, cu.cpu())):
        with pytest.raises(ValueError):
            sa.packed_forward(*bad)
    with pytest.raises(sa.SageError):
        sa.packed_forward(values(70, 3, 64), values(70, 2, 64), values(70, 2, 64), cu)
    with pytest.raises(sa.SageError):   # a row that every token shares
        sa.packed_backward(q, k, v, o, lse, do[:1].expand(70, 2, 64), cu)
    with pytest.raises(sa.SageError):   # the forward's workspace
        sa.packed_backward(q, k, v, o, lse, do, cu, ws=ws)
    dq = torch.empty_like(q)
    with pytest.raises(sa.SageError):
        sa.packed_backward(q, k, v, o, lse, do, cu, dk=dq[:, :1], dv=dq[:, :1])
    with pytest.raises(sa.SageError):
        sa.packed_backward(q, k, v, o, lse, do, cu, dq=do)
    t, _, _ = table(64, False)
    for bad in (dict(q=q.half()), dict(q=q, k=k[1:]), dict(q=q[None], k=k), dict(q=q, start=cu[:2]), dict(q=q[None], cu_seqlens=cu),
                dict(q=q, positions=cu), dict(q=q, q_out=q.float()), dict(q=q, cu_seqlens=cu.long())):
        with pytest.raises(ValueError):
            sa.rotary(t, **bad)
    for bad in (dict(q=q, k=q[:, :1], q_out=q, k_out=q[:, :1]), dict(q=q, q_out=o[:1].expand(70, 2, 64))):
        with pytest.raises(sa.SageError):
            sa.rotary(t, **bad)
    torch.cuda.synchronize()


# ------------------------------------------------------------------- streams, strides

def test_two_streams_at_once():
    q, k, v, do, cu = ref.inputs([700, 200, 1], 4, 2, 128)
    q2, k2, v2, do2, cu2 = ref.inputs([1500], 4, 2, 64, seed=1)
    t, _, _ = table(64, False)

    def step(q, k, v, do, cu, stream, ws=None):
        q, k = sa.rotary(t, q, k, cu_seqlens=cu, stream=stream)
        o, lse = sa.packed_forward(q, k, v, cu, stream=stream, ws=ws)
        dq, dk, dv = sa.packed_backward(q, k, v, o, lse, do, cu, stream=stream, ws=ws)
        return (o, lse, *sa.rotary_backward(t, dq, dk, cu_seqlens=cu, stream=stream), dv)

    want = step(q, k, v, do, cu, None), step(q2, k2, v2, do2, cu2, None)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    ws = sa.alloc_packed_ws(901, 3, 4, 2, 128, backward=True), sa.alloc_packed_ws(1500, 1, 4, 2, 64, backward=True)
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        got.append((step(q, k, v, do, cu, streams[0], ws[0]), step(q2, k2, v2, do2, cu2, streams[1], ws[1])))
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            for x, y in zip(g, w):
                assert torch.equal(x, y)


@pytest.mark.parametrize("far", ["token", "head"])
def test_strides_past_32_bits(far):
    """Tensors whose last rows lie more than 2^31 elements behind their first."""
    lens, H, Hkv, D = [200, 99], 3, 3, 64
    T = sum(lens)
    q, k, v, do, cu = ref.inputs(lens, H, Hkv, D)
    o, lse = sa.packed_forward(q, k, v, cu)
    grads = sa.packed_backward(q, k, v, o, lse, do, cu)
    t, _, _ = table(64, False)
    turn = sa.rotary(t, q, k, cu_seqlens=cu)
    # (one buffer, a slice of its inner axis for each tensor)
    if far == "token":
        memory = torch.empty((T, 7_500_032), dtype=torch.bfloat16, device="cuda")
        part = [memory[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(10)]
    else:
        memory = torch.empty((H, 1_100_000_000 // 64 * 64), dtype=torch.bfloat16, device="cuda")
        part = [memory[:, i * T * D:(i + 1) * T * D].unflatten(1, (T, D)).transpose(0, 1) for i in range(10)]
    assert max(part[0].stride()) * (part[0].shape[0 if far == "token" else 1] - 1) > 2 ** 31
    for x, y in zip(part, (q, k, v, do)):
        x.copy_(y)
    for x in part[4:]:
        x.zero_()
    Q, K, V, dO, O, dQ, dK, dV, tq, tk = part
    sa.packed_forward(Q, K, V, cu, o=O, lse=lse)
    assert torch.equal(O, o)
    sa.packed_backward(Q, K, V, O, lse, dO, cu, dq=dQ, dk=dK, dv=dV)
    for x, y in zip((dQ, dK, dV), grads):
        assert torch.equal(x, y)
    sa.rotary(t, Q, K, cu_seqlens=cu, q_out=tq, k_out=tk)
    assert torch.equal(tq, turn[0]) and torch.equal(tk, turn[1])


def test_rotary_entries_out_of_order_stay_in_bounds():
    """Any entries: the tokens that are turned are turned by some position, the others left."""
    t, _, _ = table(64, False)
    q = values(50, 2, 64)
    for entries in ([0, 2 ** 31 - 1, -5, 50], [-2 ** 31, 20, 10, 2 ** 31 - 1], [60, 40, 20, 0], [0, 0, 0, 0]):
        out = torch.full_like(q, 7.0)
        sa.rotary(t, q, cu_seqlens=ints(*entries), start=ints(2 ** 31 - 1, -2 ** 31, 5), q_out=out)
        size = q.double().unflatten(2, (2, 32)).norm(dim=2)
        now = out.double().unflatten(2, (2, 32)).norm(dim=2)
        left = (out == 7).all(-1).all(-1)
        assert ((now - size).abs() <= size * 2.0 ** -7)[~left].all()
        if entries == [0, 0, 0, 0]:
            assert left.all()
