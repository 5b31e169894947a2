"""Bounded device waits: a wait that nothing satisfies gives up, records
SAGE_ERR_TIMEOUT in the workspace status word and leaves the context usable."""
import threading

import pytest
import torch

import bit_trainable_attention_sagebwd_gb300 as sa

pytestmark = pytest.mark.gpu


def test_bounded_wait_reports_timeout_and_context_survives():
    ws = sa.alloc_ws(1, 1, 128, 64)
    ws.zero_()
    s = sa._stream_ptr()
    assert sa.sage_attn_selftest_wait(sa._ptr(ws), 1_000_000, s) == sa.SAGE_OK  # 1 ms budget
    assert sa.get_status(ws) == sa.SAGE_ERR_TIMEOUT
    assert sa.get_status(ws) == sa.SAGE_OK  # read clears the word
    x = torch.ones(1024, device="cuda")
    assert float(x.sum()) == 1024.0  # the context still works


@pytest.mark.parametrize("budget_ns", [0, 1, 1000, 100_003, 3_000_000])
def test_a_warp_gives_a_wait_up_as_one(budget_ns):
    """Lanes whose budgets differ: the wait ends for all of them (another status than the timeout's: not for all)."""
    ws = sa.alloc_ws(1, 1, 128, 64)
    ws.zero_()
    for _ in range(20):
        assert sa.sage_attn_selftest_wait(sa._ptr(ws), budget_ns, sa._stream_ptr()) == sa.SAGE_OK
        assert sa.get_status(ws) == sa.SAGE_ERR_TIMEOUT


def test_unsupported_shapes_raise():
    q = torch.zeros(1, 1, 128, 96, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(sa.SageError):
        sa.quantize(q, q, q)


def test_the_first_call_of_a_host_thread():
    """Each entry point that makes tensor maps as the first use of the GPU by its thread, on given buffers: the
    same bits as from this thread."""
    B, H, N, D = 1, 2, 256, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, do = (torch.randn((B, H, N, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(4))
    ws = sa.quantize(q, k, v)
    c = sa.kv_cache(8, H, D, B, 8)
    n = torch.full((B,), N, dtype=torch.int32, device="cuda")
    sa.kv_append(c, k, v, sa.kv_extend(c, n), n)
    one = q[:, :, :1].contiguous()

    def buffers():
        new = {x: torch.zeros_like(q) for x in ("o", "dq", "dk", "dv", "kv_o")}
        new |= {x: torch.zeros((B, H, N), dtype=torch.float32, device="cuda") for x in ("lse", "kv_lse")}
        return new | dict(one_o=torch.zeros_like(one), one_lse=torch.zeros((B, H, 1), dtype=torch.float32, device="cuda"))

    here, there = buffers(), buffers()
    kv_ws, one_ws, bws = sa.alloc_kv_ws(c, B, H, N), sa.alloc_kv_ws(c, B, H, 1), sa.alloc_bwd_ws(B, H, N, D)
    calls = {
        "forward": lambda x: sa.forward(ws, B, H, N, D, True, o=x["o"], lse=x["lse"]),
        "backward": lambda x: sa.backward(q, k, v, x["o"], x["lse"], do, ws, True, bwd_ws=bws, dq=x["dq"], dk=x["dk"], dv=x["dv"]),
        "one token": lambda x: sa.kv_attention(one, c, o=x["one_o"], lse=x["one_lse"], ws=one_ws),
        "many rows": lambda x: sa.kv_attention(q, c, o=x["kv_o"], lse=x["kv_lse"], ws=kv_ws),
    }
    failed = []

    def first(name):
        try:
            calls[name](there)
        except Exception as e:
            failed.append((name, e))

    for name in calls:
        calls[name](here)
        torch.cuda.synchronize()
        t = threading.Thread(target=first, args=(name,))
        t.start()
        t.join()
        torch.cuda.synchronize()
    assert not failed, failed
    for x in here:
        if x == "dq":  # (summed with atomics: in any order)
            assert torch.allclose(here[x].float(), there[x].float(), rtol=2 ** -7, atol=1e-5)
        else:
            assert torch.equal(here[x], there[x]), x
    assert sa.get_status(ws) == sa.SAGE_OK and sa.get_status(c.status) == sa.SAGE_OK
