"""Attention over packed sequences on the GPU against 64-bit references."""
import math

import pytest
import torch

import bit_trainable_attention_sagebwd_gb300 as sa
import packed_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def fp32_default():
    """torch's default type as it is for a user: another module of the run may have changed it."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


# lengths, H, Hkv, D, causal
CASES = [
    ([1], 1, 1, 64, True),
    ([1], 8, 2, 128, False),
    ([0, 5, 0, 0, 1, 16, 17, 0], 4, 4, 128, True),
    ([127, 128, 129], 2, 2, 128, True),
    ([127, 128, 129, 255, 256, 257], 2, 1, 64, False),
    ([31, 32, 33, 63, 64, 65], 16, 4, 128, True),          # a row tile of 32 tokens
    ([300, 1, 77], 7, 1, 128, True),                       # of 18 tokens, 126 rows
    ([300, 1, 77], 15, 3, 64, False),                      # of 25 tokens, 125 rows
    ([90, 200], 128, 1, 64, True),                         # of one token
    ([90, 200], 96, 1, 128, False),                        # of one token, 96 rows
    ([1000, 3, 700], 8, 2, 128, True),
    ([1000, 3, 700], 4, 4, 64, True),
    ([2100], 6, 2, 128, True),
    ([2100, 1111], 2, 2, 128, False),
    ([1] * 700, 4, 2, 64, True),                           # more sequences than the kernels keep sums for
    ([3, 0] * 700 + [200], 2, 1, 128, True),
]
IDS = [f"{len(c[0])}x{max(c[0])}_h{c[1]}_{c[2]}_d{c[3]}_{'causal' if c[4] else 'full'}" for c in CASES]


def forward_checked(q, k, v, cu, causal, scale=None, **kw):
    D = q.shape[2]
    ws = sa.alloc_packed_ws(q.shape[0], cu.numel() - 1, q.shape[1], k.shape[1], D)
    o, lse = sa.packed_forward(q, k, v, cu, causal=causal, sm_scale=scale, ws=ws, **kw)
    assert sa.get_status(ws) == sa.SAGE_OK
    b, e = int(cu[0]), int(cu[-1])
    want_o, want_lse, o_tol, lse_tol = ref.forward(q, k, v, cu, causal, D ** -0.5 if scale is None else scale)
    ref.check(o[b:e], want_o[b:e], o_tol[b:e], "O")
    ref.check(lse[:, b:e], want_lse[:, b:e], lse_tol[:, b:e], "LSE")
    return o, lse


@pytest.mark.parametrize("lens,H,Hkv,D,causal", CASES, ids=IDS)
def test_forward(lens, H, Hkv, D, causal):
    q, k, v, _, cu = ref.inputs(lens, H, Hkv, D)
    forward_checked(q, k, v, cu, causal)


@pytest.mark.parametrize("D", [64, 128])
def test_rows_around_the_sequences_are_left(D):
    """NaN around the sequences is neither read into a result nor written over."""
    q, k, v, _, cu = ref.inputs([40, 0, 129, 3], 4, 2, D, before=5, behind=200)
    o = torch.full((cu[-1] + 200, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, o.shape[0]), 7.0, device="cuda")
    forward_checked(q, k, v, cu, True, o=o, lse=lse)
    b, e = int(cu[0]), int(cu[-1])
    assert (o[:b] == 7).all() and (o[e:] == 7).all() and (lse[:, :b] == 7).all() and (lse[:, e:] == 7).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("causal", [True, False])
def test_values_that_are_not_finite_stay_in_their_sequence(bad, causal):
    lens = [100, 37, 5, 150, 33]
    q, k, v, _, cu = ref.inputs(lens, 4, 1, 128)
    clean = sa.packed_forward(q, k, v, cu, causal=causal)
    at = cu.tolist()
    for s in (1, 3):
        for x in (q, k, v):
            x[at[s]:at[s + 1]] = bad
    o, lse = sa.packed_forward(q, k, v, cu, causal=causal)
    for s in range(5):
        rows = slice(at[s], at[s + 1])
        if s in (1, 3):
            assert not torch.isfinite(o[rows]).any()
        else:
            assert torch.equal(o[rows], clean[0][rows]) and torch.equal(lse[:, rows], clean[1][:, rows])


def test_a_query_of_nan_gives_nan():
    q, k, v, _, cu = ref.inputs([150], 4, 2, 64)
    q[17, 1, 5] = math.nan
    o, lse = sa.packed_forward(q, k, v, cu)
    assert torch.isnan(o[17, 1]).all() and torch.isnan(lse[1, 17])
    bad = torch.isnan(o).any(-1)
    assert int(bad.sum()) == 1 and int(torch.isnan(lse).sum()) == 1


@pytest.mark.parametrize("gain,scale", [(30.0, None), (300.0, 1.0), (1.0, 1e-6), (1e-3, 5.0)])
def test_logits_of_any_size(gain, scale):
    q, k, v, _, cu = ref.inputs([300, 200], 2, 1, 128, gain=gain)
    forward_checked(q, k, v, cu, True, scale)


@pytest.mark.parametrize("grow", [1.0, -1.0])
def test_a_maximum_that_keeps_moving(grow):
    """Keys whose logits grow (or fall) along the sequence: the running reference is raised tile after tile."""
    q, k, v, _, cu = ref.inputs([1500], 2, 2, 64)
    q[:] = 1.0
    k[:] = (torch.arange(1500, device="cuda")[:, None, None] * (0.05 * grow)).to(torch.bfloat16)
    forward_checked(q, k, v, cu, True)
    forward_checked(q, k, v, cu, False)


@pytest.mark.parametrize("layout", ["fused", "heads first", "every other token"])
def test_strides(layout):
    H, Hkv, D, lens = 6, 2, 64, [70, 200, 1]
    q, k, v, _, cu = ref.inputs(lens, H, Hkv, D)
    plain = sa.packed_forward(q, k, v, cu)
    T = q.shape[0]
    if layout == "fused":
        x = torch.cat((q, k, v), 1)
        q2, k2, v2 = x.split((H, Hkv, Hkv), 1)
        o = torch.zeros((T, H + 3, D), dtype=torch.bfloat16, device="cuda")[:, 2:2 + H]
    elif layout == "heads first":
        q2, k2, v2 = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
        o = torch.zeros((H, T, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    else:
        q2, k2, v2 = (torch.stack((x, torch.full_like(x, math.nan)), 1).flatten(0, 1)[::2] for x in (q, k, v))
        o = torch.zeros((2 * T, H, D), dtype=torch.bfloat16, device="cuda")[::2]
    got = sa.packed_forward(q2, k2, v2, cu, o=o)
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


@pytest.mark.parametrize("entries", [[0, 50, 110, 181], [-1, 50, 110, 180], [0, 2 ** 31 - 1, 110, 180], [-2 ** 31, -5, 110, 180],
                                     [0, 50, 40, 180], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0]], ids=str)
def test_sequences_out_of_order_or_range_are_left_out(entries):
    q, k, v, _, _ = ref.inputs([180], 2, 1, 64)
    ws = sa.alloc_packed_ws(180, 3, 2, 1, 64)
    o = torch.full_like(q, 7.0)
    sa.packed_forward(q, k, v, torch.tensor(entries, dtype=torch.int32, device="cuda"), o=o, ws=ws)
    assert sa.get_status(ws) == sa.SAGE_ERR_INVALID_ARG
    assert sa.get_status(ws) == sa.SAGE_OK
    times = torch.zeros(180, dtype=torch.int32)
    good = [(b, e) for b, e in zip(entries, entries[1:]) if 0 <= b <= e <= 180]
    for b, e in good:
        times[b:e] += 1
    for b, e in good:
        want, _ = sa.packed_forward(q[b:e], k[b:e], v[b:e], torch.tensor([0, e - b], dtype=torch.int32, device="cuda"))
        once = (times[b:e] == 1).cuda()
        assert torch.equal(o[b:e][once], want[once])
    assert (o[(times == 0).cuda()] == 7).all()


def test_captured_with_other_lengths():
    """One captured call, replayed after cu_seqlens has changed."""
    q, k, v, _, cu = ref.inputs([300, 200, 100], 4, 2, 128)
    ws = sa.alloc_packed_ws(600, 3, 4, 2, 128)
    o, lse = torch.zeros_like(q), torch.zeros((4, 600), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sa.packed_forward(q, k, v, cu, o=o, lse=lse, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sa.packed_forward(q, k, v, cu, o=o, lse=lse, ws=ws)
    for lens in ([0, 599, 1], [200, 200, 200], [0, 0, 3]):
        cu.copy_(torch.tensor([0] + lens).cumsum(0).to(torch.int32))
        o.fill_(7.0)
        g.replay()
        want = sa.packed_forward(q, k, v, cu)
        n = sum(lens)
        assert torch.equal(o[:n], want[0][:n]) and torch.equal(lse[:, :n], want[1][:, :n]) and (o[n:] == 7).all()


def test_the_same_bits_every_time():
    q, k, v, _, cu = ref.inputs([3000, 500, 1], 8, 2, 128)
    first = sa.packed_forward(q, k, v, cu)
    for _ in range(5):
        again = sa.packed_forward(q, k, v, cu)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_on_a_stream():
    q, k, v, _, cu = ref.inputs([300, 200], 4, 2, 128)
    want = sa.packed_forward(q, k, v, cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = sa.packed_forward(q, k, v, cu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------- gradients

def backward_checked(q, k, v, do, cu, causal, scale=None, **kw):
    D = q.shape[2]
    o, lse = sa.packed_forward(q, k, v, cu, causal=causal, sm_scale=scale)
    ws = sa.alloc_packed_ws(q.shape[0], cu.numel() - 1, q.shape[1], k.shape[1], D, backward=True)
    got = dict(zip(("dq", "dk", "dv"), sa.packed_backward(q, k, v, o, lse, do, cu, causal=causal, sm_scale=scale, ws=ws, **kw)))
    assert sa.get_status(ws) == sa.SAGE_OK
    want, tol = ref.backward(q, k, v, o, lse, do, cu, causal, D ** -0.5 if scale is None else scale)
    b, e = int(cu[0]), int(cu[-1])
    for n in got:
        ref.check(got[n][b:e], want[n][b:e], tol[n][b:e], n)
    return o, lse, got


@pytest.mark.parametrize("lens,H,Hkv,D,causal", CASES, ids=IDS)
def test_backward(lens, H, Hkv, D, causal):
    q, k, v, do, cu = ref.inputs(lens, H, Hkv, D, seed=1)
    backward_checked(q, k, v, do, cu, causal)


@pytest.mark.parametrize("D", [64, 128])
def test_gradients_of_rows_around_the_sequences_are_left(D):
    q, k, v, do, cu = ref.inputs([40, 0, 129, 3], 4, 2, D, before=5, behind=200)
    kw = {"d" + n: torch.full_like(x, 7.0) for n, x in (("q", q), ("k", k), ("v", v))}
    _, _, got = backward_checked(q, k, v, do, cu, True, **kw)
    b, e = int(cu[0]), int(cu[-1])
    for x in got.values():
        assert (x[:b] == 7).all() and (x[e:] == 7).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G", [1, 3, 4])
def test_gradients_that_are_not_finite_stay_in_their_sequence(bad, causal, G):
    lens = [100, 37, 5, 150, 33]
    q, k, v, do, cu = ref.inputs(lens, G, 1, 128)
    o, lse = sa.packed_forward(q, k, v, cu, causal=causal)
    clean = sa.packed_backward(q, k, v, o, lse, do, cu, causal=causal)
    at = cu.tolist()
    for s in (1, 3):
        for x in (q, k, v, o, do):
            x[at[s]:at[s + 1]] = bad
        lse[:, at[s]:at[s + 1]] = bad
    got = sa.packed_backward(q, k, v, o, lse, do, cu, causal=causal)
    for s in (0, 2, 4):
        rows = slice(at[s], at[s + 1])
        for x, y in zip(got, clean):
            assert torch.equal(x[rows], y[rows])


@pytest.mark.parametrize("gain,scale", [(30.0, None), (1.0, 1e-6), (1e-3, 5.0)])
def test_gradients_at_logits_of_any_size(gain, scale):
    q, k, v, do, cu = ref.inputs([300, 200], 2, 1, 128, gain=gain)
    backward_checked(q, k, v, do, cu, True, scale)


@pytest.mark.parametrize("D,causal", [(64, True), (128, False)])
def test_gradients_against_differences(D, causal):
    """Sum dO O of the 64-bit forward along a direction."""
    lens, H, Hkv = [33, 70], 4, 2
    q, k, v, do, cu = ref.inputs(lens, H, Hkv, D, seed=3)
    o, lse = sa.packed_forward(q, k, v, cu, causal=causal)
    grads = sa.packed_backward(q, k, v, o, lse, do, cu, causal=causal)
    _, tol = ref.backward(q, k, v, o, lse, do, cu, causal, D ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = [y.double() for y in (q, k, v)]
    for n, name in enumerate(("dq", "dk", "dv")):
        way = torch.randn(x[n].shape, dtype=torch.float64, device="cuda", generator=g)
        h = 1e-5

        def loss(step):
            y = list(x)
            y[n] = x[n] + step * way
            return (do.double() * ref.forward(*y, cu, causal, D ** -0.5)[0]).sum()

        slope = (loss(h) - loss(-h)) / (2 * h)
        # each gradient's bound along the way; O's rounding enters delta; the difference itself is good to h^2
        delta_off = ref.BF16 * (do.double() * o.double()).abs().sum() * 10 * D ** -0.5 * way.abs().max() if n < 2 else 0.0
        most = (tol[name] * way.abs()).sum() + delta_off + 1e-6
        assert abs(float((grads[n].double() * way).sum() - slope)) <= float(most), name


@pytest.mark.parametrize("layout", ["fused", "heads first"])
def test_strides_of_the_gradients(layout):
    H, Hkv, D, lens = 6, 2, 64, [70, 200, 1]
    q, k, v, do, cu = ref.inputs(lens, H, Hkv, D)
    o, lse = sa.packed_forward(q, k, v, cu)
    plain = sa.packed_backward(q, k, v, o, lse, do, cu)
    if layout == "fused":
        x = torch.cat((q, k, v), 1)
        q2, k2, v2 = x.split((H, Hkv, Hkv), 1)
        dx = torch.zeros_like(x)
        dq, dk, dv = dx.split((H, Hkv, Hkv), 1)
        o2, do2 = o, do
    else:
        q2, k2, v2, o2, do2 = (y.transpose(0, 1).contiguous().transpose(0, 1) for y in (q, k, v, o, do))
        dq, dk, dv = (torch.zeros_like(y) for y in (q2, k2, v2))
    got = sa.packed_backward(q2, k2, v2, o2, lse, do2, cu, dq=dq, dk=dk, dv=dv)
    for x, y in zip(got, plain):
        assert torch.equal(x, y)


def test_the_same_gradients_every_time():
    q, k, v, do, cu = ref.inputs([3000, 500, 1], 8, 2, 128)
    o, lse = sa.packed_forward(q, k, v, cu)
    first = sa.packed_backward(q, k, v, o, lse, do, cu)
    for _ in range(5):
        for x, y in zip(first, sa.packed_backward(q, k, v, o, lse, do, cu)):
            assert torch.equal(x, y)


def test_a_captured_step():
    """Forward and backward in one graph, replayed with other values and lengths."""
    q, k, v, do, cu = ref.inputs([300, 200, 100], 4, 2, 128)
    ws = sa.alloc_packed_ws(600, 3, 4, 2, 128, backward=True)
    o, lse = torch.zeros_like(q), torch.zeros((4, 600), device="cuda")
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))

    def step():
        sa.packed_forward(q, k, v, cu, o=o, lse=lse, ws=ws)
        sa.packed_backward(q, k, v, o, lse, do, cu, dq=dq, dk=dk, dv=dv, ws=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n, lens in enumerate(([0, 599, 1], [200, 200, 200], [0, 0, 3])):
        cu.copy_(torch.tensor([0] + lens).cumsum(0).to(torch.int32))
        q.copy_(ref.inputs([600], 4, 2, 128, seed=n)[0])
        g.replay()
        rows = sum(lens)
        want = sa.packed_forward(q, k, v, cu)
        grads = sa.packed_backward(q, k, v, *want, do, cu)
        assert torch.equal(o[:rows], want[0][:rows])
        for x, y in zip((dq, dk, dv), grads):
            assert torch.equal(x[:rows], y[:rows])
