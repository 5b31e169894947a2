"""Orders between kernels and between threads that the memory model asks for and no run can show, read from the sources."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_trainable_attention_sagebwd_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def closed(text, at, pair):
    """The place behind the bracket that closes the one before `at`."""
    depth = 1
    while depth:
        depth += {pair[0]: 1, pair[1]: -1}.get(text[at], 0)
        at += 1
    return at


def body(text, name):
    """The text between the braces of function `name`'s definition."""
    for m in re.finditer(r"\b%s\s*\(" % name, text):
        at = closed(text, m.end(), "()")
        opens = re.match(r"\s*(const\s*)?\{", text[at:])
        if opens:
            return text[at + opens.end():closed(text, at + opens.end(), "{}") - 1]
    raise AssertionError(f"{name}: no definition")


def kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = source(os.path.basename(path))
        for m in re.finditer(r"__global__\s+void\s+(__launch_bounds__\()?", text):
            at = closed(text, m.end(), "()") if m.group(1) else m.end()
            name = re.match(r"\s*(\w+)", text[at:]).group(1)
            code = body(text, name)
            if "pdl_" in code:
                yield pytest.param(code, id=name)


# what reads memory that a predecessor may have written
READS = r"__ldg\(|__ldcg\(|tma_load_3d\(|bulk_load\(|prefix_of\w*<|prefix_of\w*\(|\brow_chunks\("


@pytest.mark.parametrize("code", list(kernels()))
def test_a_kernel_waits_for_its_predecessor_before_it_reads_and_lets_others_in(code):
    wait = re.search(r"\bpdl_wait(_unless)?\(", code)
    assert wait, "no wait"
    trigger = re.search(r"\bpdl_trigger\(", code)
    assert trigger is None or wait.start() < trigger.start(), "lets its dependents in before its own wait"
    first = re.search(READS, code)
    assert first is None or wait.start() < first.start(), f"{first.group()} before the wait"


def test_inputs_staged_before_the_wait_come_from_before_an_ordinary_operation():
    """The quantize kernels stage Q, K and V before their waits: the clearing in front of them, which is no programmatic
    launch, comes behind all of what wrote these."""
    launch = body(source("quantize.cu"), "launch_quantize")
    assert launch.index("cudaMemsetAsync(") < launch.index("launch_pdl(")


def test_a_kernel_that_does_not_wait_is_told_and_keeps_the_order():
    text = source("packed_bwd.cu")
    dkv, dq = body(text, "packed_dkv_kernel"), body(text, "packed_dq_kernel")
    assert dkv.index("pdl_wait(") < dkv.index("pdl_tell(") < dkv.index("__syncthreads()") < dkv.index("pdl_trigger(")
    assert dq.index("pdl_wait_unless(") < dq.index("pdl_wait(") < dq.index("kTermsTold, 0)")
    # the ordinary wait is the last thing but that
    assert not re.search(READS, dq[dq.index("pdl_wait("):])
    ptx = source("ptx.cuh")
    assert "st.release.gpu" in body(ptx, "pdl_tell")
    told = body(ptx, "pdl_wait_unless")
    assert told.index("ld.acquire.gpu") < told.index("pdl_wait()") < told.index("fence.proxy.async.global")


def test_the_sums_of_all_warps_go_out_with_the_count():
    """Of a join only the lane that counts releases what it has learned of: a fence between its wait for the other warps
    and the count, one between the count and its word to them, and theirs before they read."""
    calls = re.findall(r"__threadfence|warp_arrive\(&written|mbar_wait_warp\(&written|atomicAdd|mbar_arrive\(&told|mbar_wait_warp\(&told"
                       r"|return ok", body(source("packed.cuh"), "was_last"))
    assert calls == ["__threadfence", "warp_arrive(&written", "mbar_wait_warp(&written", "__threadfence", "atomicAdd",
                     "__threadfence", "mbar_arrive(&told", "mbar_wait_warp(&told", "__threadfence", "return ok"]
