"""More of packed attention and rotary positions without a GPU: the device status words, calls without tokens, small scales,
the table's fractions, and the 64-bit reference of the gradients against differences."""
import decimal
import math
import os
import re

import pytest
import torch

import packed_ref as ref
import packed_rests as rests
import bit_trainable_attention_sagebwd_gb300 as sa
from bit_trainable_attention_sagebwd_gb300 import rotary_positions
from test_packed_host import backward, lib  # noqa: F401

CSRC = os.path.join(os.path.dirname(os.path.abspath(sa.__file__)), "csrc")


def test_a_wait_that_ran_out_hides_behind_no_other_report():
    """The status word keeps the largest code; a workspace whose counters may not be zero has to say so, whatever
    entries were out of range."""
    code = {}
    for name in ("ptx.cuh", "kv.h", "packed.cuh"):
        with open(os.path.join(CSRC, name)) as f:
            code |= {n: int(v) for n, v in re.findall(r"\b(kDev\w+) = (\d+)", f.read())}
    assert set(code) == {"kDevOk", "kDevSetup", "kDevTimeout", "kDevPages", "kDevIndex", "kDevSequence"}
    assert code["kDevOk"] == 0 and code["kDevSequence"] == code["kDevIndex"]
    for x in ("kDevSetup", "kDevTimeout"):
        assert all(code[x] > code[y] for y in ("kDevPages", "kDevIndex", "kDevSequence"))


@pytest.mark.parametrize("scale", [1e-45, 1e-38, 5e-38, 7e-37])
def test_gradients_at_scales_that_LSE_cannot_be_divided_by(lib, scale):
    """(Below 5e-38 LSE / sm_scale was infinite for some 700 keys, and every P 0.)"""
    assert backward(sm_scale=scale) == sa.SAGE_ERR_UNSUPPORTED


PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")
FREQUENCIES = [1.0, -1.0, 0.5, 1e-4, 10000.0 ** (-126 / 128), 500000.0 ** (-2 / 128), 1e-12, 1e-300, 0.0, math.pi, 2 * math.pi, -7.25, 6.283,
               1e5, -1e9, 2.0 ** 60]


@pytest.mark.parametrize("f", FREQUENCIES, ids=str)
def test_fractions_of_a_turn_are_the_nearest(f):
    """Against 100 digits: what a table holds is off by half of 2^-64 turns at most, whole turns apart."""
    with decimal.localcontext(prec=160):
        exact = decimal.Decimal(f) / (2 * PI) * 2 ** 64
        got = rotary_positions._turns(f)
        off = (exact - got) % 2 ** 64
        assert -2 ** 63 <= got < 2 ** 63 and min(off, 2 ** 64 - off) <= decimal.Decimal("0.5000001")


def test_the_digits_of_pi():
    with decimal.localcontext(prec=160):
        for bits in (64, 300, 330):
            off = PI * 2 ** bits - rotary_positions._pi(bits)
            assert -1 <= off <= 2


# ------------------------------------------------------------------- what the GPU's results are compared with

@pytest.mark.parametrize("D,causal,G", [(64, True, 2), (128, False, 3)])
def test_the_reference_gradients_against_differences(D, causal, G):
    """Sum dO O of the 64-bit forward along a direction at random: the reference's gradients, from its own O and LSE."""
    Hkv, scale = 2, D ** -0.5
    *x, do, cu = ref.inputs([33, 1, 70], G * Hkv, Hkv, D, seed=3, device="cpu")
    x, do = [y.double() for y in x], do.double()
    o, lse, _, _ = ref.forward(*x, cu, causal, scale)
    grads, _ = ref.backward(*x, o, lse, do, cu, causal, scale)
    g = torch.Generator().manual_seed(5)
    for n, name in enumerate(("dq", "dk", "dv")):
        way, h = torch.randn(x[n].shape, dtype=torch.float64, generator=g), 1e-4

        def loss(step):
            y = list(x)
            y[n] = x[n] + step * way
            return (do * ref.forward(*y, cu, causal, scale)[0]).sum()

        # (off by h^2 of the third derivative, and by 64-bit rounding over h)
        slope = float((loss(h) - loss(-h)) / (2 * h))
        assert abs(float((grads[name] * way).sum()) - slope) <= 1e-6 * float(grads[name].norm() * way.norm()), name


def emulated(q, k, v, o, lse, do, cu, causal, low):
    """dQ with dS rounded to bf16 and what `low` makes of the roundings' rests."""
    D, out = q.shape[2], torch.zeros_like(q)
    for b, e in zip(cu.tolist(), cu.tolist()[1:]):
        for h in range(q.shape[1]):
            kh, doh = k[b:e, 0].double(), do[b:e, h].double()
            p = torch.exp(ref._logits(q[b:e, h].double(), kh, causal, D ** -0.5) - lse[h, b:e, None].double())
            ds = p * (doh @ v[b:e, 0].double().T - (doh * o[b:e, h].double()).sum(-1, keepdim=True))
            high = ds.to(torch.bfloat16).double()
            out[b:e, h] = (D ** -0.5 * (high + low((ds - high) * rests.carried(e - b))) @ kh).to(torch.bfloat16)
    return out


@pytest.mark.parametrize("D,causal", [(64, False), (64, True), (128, False), (128, True)])
def test_the_check_of_the_rests_sees_what_is_wrong(D, causal):
    q, k, v, do, cu = rests.inputs(2, D, 7, "cpu")
    o, lse, _, _ = ref.forward(q, k, v, cu, causal, D ** -0.5)
    o, lse = o.to(torch.bfloat16), lse.float()
    want = ref.backward(q, k, v, o, lse, do, cu, causal, D ** -0.5)[0]["dq"]

    def dq(low):
        return emulated(q, k, v, o, lse, do, cu, causal, low)

    rests.check(dq(lambda x: x.to(torch.bfloat16).double()), want, cu)
    at = cu.tolist()
    for wrong in (lambda x: 0 * x, lambda x: -x, lambda x: x.roll(8, 1)):
        got = dq(wrong)
        for n, b, e in zip(rests.LENS, at, at[1:]):
            off = float((got[b:e].double() - want[b:e]).norm() / want[b:e].norm())
            assert off > rests.MOST, (n, off)
