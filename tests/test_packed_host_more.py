"""More of packed attention and rotary positions without a GPU: the device status words, calls without tokens, small scales,
the table's fractions, and the 64-bit reference of the gradients against differences."""
import os
import re

import pytest

import bit_trainable_attention_sagebwd_gb300 as sa
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
