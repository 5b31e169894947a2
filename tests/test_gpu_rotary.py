"""Rotary positions on the GPU against complex numbers in 64 bits."""
import math

import pytest
import torch

import bit_trainable_attention_sagebwd_gb300 as sa

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def fp32_default():
    """torch's default type as it is for a user: another module of the run may have changed it."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


BF16 = torch.finfo(torch.bfloat16).eps / 2


def turned(x, pos, freq, rot, interleaved, gain, inverse):
    """x [.., tokens, D] with positions pos [.., tokens], and the bound of the library's error: bf16's rounding of the
    result, and of the pair's size fp32's roundings (angle, sine, cosine, two products and a sum: 2^-24 each, the angle in
    units of pi), beside the angle's own in these 64 bits."""
    y = x.double().clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    angle = pos.double()[..., None] * freq.to(x.device)
    z = torch.complex(y[..., a], y[..., b])
    w = z * torch.polar(torch.full_like(angle, gain), -angle if inverse else angle)
    y[..., a], y[..., b] = w.real, w.imag
    off = torch.zeros_like(y)
    size = z.abs() * gain * (2.0 ** -20 + angle.abs() * 2.0 ** -52)
    off[..., a], off[..., b] = size, size
    return y, off + BF16 * 1.01 * y.abs()


def check(got, want):
    y, off = want
    bad = ~((got.double() - y).abs() <= off)
    assert not bad.any(), f"{int(bad.sum())} elements, the first at {bad.nonzero()[0].tolist()}"


def values(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def table(rot, interleaved, **kw):
    f, gain = sa.rotary_frequencies(rot, **kw)
    return sa.rotary_table(rot, interleaved=interleaved, **kw), torch.tensor(f, dtype=torch.float64), gain


SCALINGS = [dict(), dict(scaling="linear", factor=3.0), dict(scaling="base", factor=8.0, base=500000.0),
            dict(scaling="ramp", factor=16.0, context=2048)]


@pytest.mark.parametrize("kw", SCALINGS, ids=lambda k: k.get("scaling", "none"))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 16), (128, 112)])
def test_new_tokens(D, rot, interleaved, kw):
    """[B, H, N, D], each sequence from its own position; there and back."""
    t, f, gain = table(rot, interleaved, **kw)
    B, H, Hkv, N = 3, 5, 2, 4
    q, k, start = values(B, H, N, D), values(B, Hkv, N, D, seed=1), ints(0, 123457, 2 ** 31 - 8)
    pos = (start[:, None].long() + torch.arange(N, device="cuda"))[:, None]
    for back in (False, True):
        got = (sa.rotary_backward if back else sa.rotary)(t, q, k, start=start)
        for x, y in zip((q, k), got):
            check(y, turned(x, pos, f, rot, interleaved, gain, back))
            assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("lens", [[1], [5, 0, 17, 0, 300], [0, 0, 1000], [1] * 100])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("begun", [False, True])
def test_packed(lens, interleaved, begun):
    """[T, H, D]: places in the sequences; rows before and behind them are left."""
    t, f, gain = table(64, interleaved, scaling="ramp", factor=4.0)
    H, Hkv, D, before, behind = 7, 3, 128, 4, 9
    T = sum(lens) + before + behind
    q, k = values(T, H, D), values(T, Hkv, D, seed=1)
    cu = (torch.tensor([0] + lens).cumsum(0) + before).to(torch.int32).cuda()
    start = torch.arange(len(lens), dtype=torch.int32, device="cuda") * 1001 if begun else None
    out = [torch.full_like(x, 7.0) for x in (q, k)]
    sa.rotary(t, q, k, cu_seqlens=cu, start=start, q_out=out[0], k_out=out[1])
    pos = torch.cat([torch.arange(n) + (1001 * s if begun else 0) for s, n in enumerate(lens)]).cuda()
    for x, y in zip((q, k), out):
        assert (y[:before] == 7).all() and (y[T - behind:] == 7).all()
        check(y[before:T - behind].transpose(0, 1), turned(x[before:T - behind].transpose(0, 1), pos, f, 64, interleaved, gain, False))


def test_many_tokens_and_few_give_the_same():
    """A batch large enough for the kernel that takes several heads a thread, and its rows alone."""
    t, *_ = table(128, False)
    q, k = values(20000, 9, 128), values(20000, 2, 128, seed=1)
    many = sa.rotary(t, q, k)
    for i in (0, 1, 777, 19999):
        one = sa.rotary(t, q[i:i + 1], k[i:i + 1], start=ints(i))
        assert torch.equal(one[0][0], many[0][i]) and torch.equal(one[1][0], many[1][i])


def test_given_positions_and_queries_alone():
    t, f, gain = table(64, True)
    q, p = values(11, 3, 64), torch.randint(-1000, 1 << 20, (11,), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    check(sa.rotary(t, q, positions=p).transpose(0, 1), turned(q.transpose(0, 1), p, f, 64, True, gain, False))
    q = values(2, 3, 5, 64)
    p = torch.randint(0, 1 << 20, (2, 5), generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    check(sa.rotary(t, q, positions=p), turned(q, p[:, None], f, 64, True, gain, False))


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_strides(interleaved):
    t, *_ = table(64, interleaved)
    T, H, Hkv, D = 50, 4, 2, 128
    x = values(T, H + 2 * Hkv, D)
    q, k, v = x.split((H, Hkv, Hkv), 1)
    want = sa.rotary(t, q.contiguous(), k.contiguous())
    kept = v.clone()
    got = sa.rotary(t, q, k, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept)
    y = values(H, T, D).transpose(0, 1)
    assert torch.equal(sa.rotary(t, y), sa.rotary(t, y.contiguous()))


def test_values_that_are_not_finite_stay_in_their_pair():
    t, *_ = table(64, False)
    q = values(4, 2, 64)
    clean = sa.rotary(t, q)
    q[2, 1, 5] = math.nan
    got = sa.rotary(t, q)
    bad = torch.isnan(got).nonzero().tolist()
    assert bad == [[2, 1, 5], [2, 1, 37]]
    assert torch.equal(got[torch.isfinite(got)], clean[torch.isfinite(got)])


def test_the_gradient_is_the_transpose():
    """Sum y' turn(x) = sum turn_backward(y') x, up to the roundings."""
    t, f, gain = table(48, True, scaling="ramp", factor=4.0)
    x, g, s = values(1, 3, 9, 64), values(1, 3, 9, 64, seed=1), ints(77)
    pos = (77 + torch.arange(9, device="cuda"))[None, None]
    y, y_off = turned(x, pos, f, 48, True, gain, False)
    dx = sa.rotary_backward(t, g, start=s)
    _, dx_off = turned(g, pos, f, 48, True, gain, True)
    most = (dx_off * x.double().abs()).sum()
    assert abs(float((g.double() * y).sum() - (dx.double() * x.double()).sum())) <= float(most)


def test_on_a_stream_and_captured():
    t, *_ = table(128, False)
    q, k, start = values(8, 4, 1, 128), values(8, 2, 1, 128, seed=1), ints(*range(8))
    want = sa.rotary(t, q, k, start=start)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = sa.rotary(t, q, k, start=start, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = [torch.empty_like(x) for x in (q, k)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sa.rotary(t, q, k, start=start, q_out=out[0], k_out=out[1])
    for step in (1, 100000):
        start += step
        g.replay()
        want = sa.rotary(t, q, k, start=start)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
