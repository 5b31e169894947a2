"""More of packed attention and rotary positions on the GPU."""
import pytest
import torch

import bit_trainable_attention_sagebwd_gb300 as sa
import packed_ref as ref
import packed_rests as rests
from test_gpu_packed import backward_checked, forward_checked, fp32_default  # noqa: F401
from test_gpu_rotary import table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_the_least_scale(D):
    """All keys weigh the same; LSE, the log of their number, is divided by 2^-120 on the way."""
    q, k, v, do, cu = ref.inputs([300, 1, 77], 4, 2, D, seed=2)
    forward_checked(q, k, v, cu, True, 2.0 ** -120)
    backward_checked(q, k, v, do, cu, True, 2.0 ** -120)


@pytest.mark.parametrize("S", [1, 3])
def test_batches_without_a_token(S):
    """A step whose share of the documents is empty: every call gives empty results."""
    q, k = (torch.empty((0, h, 64), dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    cu = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    t, _, _ = table(64, False)
    ws = sa.alloc_packed_ws(0, S, 4, 2, 64, backward=True)
    for given in (None, ws):
        tq, tk = sa.rotary(t, q, k, cu_seqlens=cu)
        o, lse = sa.packed_forward(tq, tk, k, cu, ws=given)
        assert o.shape == q.shape and o.dtype == q.dtype and lse.shape == (4, 0) and lse.dtype == torch.float32
        grads = sa.packed_backward(tq, tk, k, o, lse, o, cu, ws=given)
        assert [x.shape for x in grads] == [q.shape, k.shape, k.shape]
        assert [x.shape for x in sa.rotary_backward(t, *grads[:2], cu_seqlens=cu)] == [q.shape, k.shape]
    assert sa.get_status(ws) == sa.SAGE_OK
    for shape in ((0, 4, 1, 64), (2, 4, 0, 64)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        assert sa.rotary(t, x, start=torch.zeros(shape[0], dtype=torch.int32, device="cuda")).shape == shape
    # refused as with tokens
    with pytest.raises(sa.SageError):
        sa.packed_forward(q[:, :3], k, k, cu, ws=ws)
    with pytest.raises(ValueError):
        sa.packed_forward(q.half(), k, k, cu)
    with pytest.raises(ValueError):
        sa.packed_backward(q, k, k, q, torch.empty((3, 0), device="cuda"), q, cu)
    with pytest.raises(sa.SageError):
        sa.rotary(t, torch.empty((0, 4, 96), dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("D,causal,G", [(64, True, 2), (128, False, 3)])
def test_gradients_along_themselves_against_differences(D, causal, G):
    """Sum dO O of the 64-bit forward along each gradient, whose slope is the gradient's square.  The library's is off by its own
    rounding (2^-8 / sqrt 3 in relative L2), P's and dS's (the same, half as much again where rows cancel) and O's in delta:
    1e-2 of the slope at most."""
    Hkv, scale = 2, D ** -0.5
    q, k, v, do, cu = ref.inputs([33, 1, 70], G * Hkv, Hkv, D, seed=3)
    o, lse = sa.packed_forward(q, k, v, cu, causal=causal)
    got = dict(zip(("dq", "dk", "dv"), sa.packed_backward(q, k, v, o, lse, do, cu, causal=causal)))
    x = [y.double() for y in (q, k, v)]
    want, _ = ref.backward(*x, *ref.forward(*x, cu, causal, scale)[:2], do, cu, causal, scale)
    for n, (name, way) in enumerate(want.items()):
        h = 1e-4 / float(way.norm())

        def loss(step):
            y = list(x)
            y[n] = x[n] + step * way
            return (do.double() * ref.forward(*y, cu, causal, scale)[0]).sum()

        slope = float((loss(h) - loss(-h)) / (2 * h))
        assert abs(float((got[name].double() * way).sum()) - slope) <= 1e-2 * slope, name


@pytest.mark.parametrize("G", [1, 2, 5])
@pytest.mark.parametrize("D,causal", [(64, False), (64, True), (128, False), (128, True)])
def test_the_rests_of_dS_go_into_dQ(D, causal, G):
    q, k, v, do, cu = rests.inputs(G, D, 7 + G, "cuda")
    o, lse = sa.packed_forward(q, k, v, cu, causal=causal)
    dq, _, _ = sa.packed_backward(q, k, v, o, lse, do, cu, causal=causal)
    rests.check(dq, ref.backward(q, k, v, o, lse, do, cu, causal, D ** -0.5)[0]["dq"], cu)


@pytest.mark.parametrize("entries", [[0, 50, 110, 181], [-1, 50, 110, 180], [0, 2 ** 31 - 1, 110, 180], [0, 50, 40, 180],
                                     [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0]], ids=str)
def test_gradients_beside_sequences_out_of_order_or_range(entries):
    """Rows of one sequence, and only of one, get what a call on that sequence alone gives."""
    q, k, v, do, cu = ref.inputs([180], 2, 1, 64)
    o, lse = sa.packed_forward(q, k, v, cu)
    out = [torch.full_like(x, 7.0) for x in (q, k, v)]
    sa.packed_backward(q, k, v, o, lse, do, torch.tensor(entries, dtype=torch.int32, device="cuda"), dq=out[0], dk=out[1], dv=out[2])
    good = [(b, e) for b, e in zip(entries, entries[1:]) if 0 <= b <= e <= 180]
    times = torch.zeros(180, dtype=torch.int32)
    for b, e in good:
        times[b:e] += 1
    for b, e in good:
        alone = torch.tensor([0, e - b], dtype=torch.int32, device="cuda")
        want = sa.packed_backward(*(x[b:e] for x in (q, k, v, o)), lse[:, b:e].contiguous(), do[b:e], alone)
        once = (times[b:e] == 1).cuda()
        for x, y in zip(out, want):
            assert torch.equal(x[b:e][once], y[once])
    for x in out:
        assert (x[(times == 0).cuda()] == 7).all()


@pytest.mark.parametrize("N", [300, 20000])
def test_turned_and_quantized_at_once(N):
    """rotary, and quantize right behind it on the same stream, which stages keys and values before it waits: the codes of
    the turned ones."""
    t, _, _ = table(128, False)
    g = torch.Generator("cuda").manual_seed(0)
    q, k, v = (torch.randn((1, 4, N, 128), device="cuda", generator=g).to(torch.bfloat16) for _ in range(3))
    tq, tk = sa.rotary(t, q, k)
    torch.cuda.synchronize()
    o, lse = sa.forward(sa.quantize(tq, tk, v), 1, 4, N, 128, causal=True)[:2]
    q2, k2 = torch.zeros_like(q), torch.zeros_like(k)
    for _ in range(10):
        q2.zero_(), k2.zero_()
        sa.rotary(t, q, k, q_out=q2, k_out=k2)
        got = sa.forward(sa.quantize(q2, k2, v), 1, 4, N, 128, causal=True)[:2]
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
