"""Attention over packed sequences and its gradients in 64 bits, from the formulas, with bounds on what the library's
roundings may change; and the inputs of the tests."""
import math

import torch

BF16, FP32 = torch.finfo(torch.bfloat16).eps / 2, torch.finfo(torch.float32).eps / 2


def inputs(lens, H, Hkv, D, seed=0, device="cuda", before=0, behind=0, gain=1.0):
    """q, k, v, do of the packed sequences and cu_seqlens; `before` and `behind` rows of NaN around them."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + before + behind

    def normal(heads, gain=1.0):
        x = (torch.randn((T, heads, D), generator=g) * gain).to(torch.bfloat16)
        x[:before] = x[T - behind:] = math.nan
        return x.to(device)

    cu = torch.tensor([0] + list(lens), dtype=torch.int64).cumsum(0) + before
    return normal(H, gain), normal(Hkv), normal(Hkv), normal(H), cu.to(torch.int32).to(device)


def _sequences(cu):
    at = cu.tolist()
    return [(b, e) for b, e in zip(at, at[1:]) if e > b]


def _logits(q, k, causal, scale):
    t = q @ k.T * scale
    return t.masked_fill(torch.ones_like(t, dtype=torch.bool).triu(1), -math.inf) if causal else t


def _slack(q, k, D, scale):
    """How far the library's logits may be from the exact ones, and 2^x from its exponent: the products are exact, each
    of D + 2 sums or products of fp32 rounds to within an ulp of the sum of the magnitudes (tensor cores may truncate);
    the exponential's result is good to 2^-22."""
    size = (q.abs() @ k.abs().T * scale).amax(-1, keepdim=True)
    return size * (D + 8) * 2 * FP32 + 2.0 ** -21


def forward(q, k, v, cu, causal, scale):
    """O, LSE and the bounds of their errors; 0 behind the sequences."""
    (T, H, D), G = q.shape, q.shape[1] // k.shape[1]
    o, o_tol = (torch.zeros(q.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    lse, lse_tol = (torch.zeros((H, T), dtype=torch.float64, device=q.device) for _ in range(2))
    for b, e in _sequences(cu):
        for h in range(H):
            qh, kh, vh = (x[b:e, i].double() for x, i in ((q, h), (k, h // G), (v, h // G)))
            t = _logits(qh, kh, causal, scale)
            p = torch.softmax(t, -1)
            slack = _slack(qh, kh, D, scale)
            o[b:e, h] = p @ vh
            lse[h, b:e] = torch.logsumexp(t, -1)
            # P rounded to bf16, the logits' errors in P and in the row sum, O rounded to bf16
            o_tol[b:e, h] = (p @ vh.abs()) * (BF16 * 1.01 + 2 * slack + 2.0 ** -20) + BF16 * 1.01 * o[b:e, h].abs()
            lse_tol[h, b:e] = slack[:, 0] + (1 + lse[h, b:e].abs()) * 2.0 ** -20
    return o, lse, o_tol, lse_tol


def backward(q, k, v, o, lse, do, cu, causal, scale):
    """dQ, dK, dV from the given O and LSE, and the bounds of their errors; 0 behind the sequences."""
    (T, H, D), G = q.shape, q.shape[1] // k.shape[1]
    out = {n: torch.zeros(x.shape, dtype=torch.float64, device=q.device) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    tol = {n: torch.zeros_like(x) for n, x in out.items()}
    for b, e in _sequences(cu):
        for h in range(H):
            n = h // G
            qh, kh, vh = (x[b:e, i].double() for x, i in ((q, h), (k, n), (v, n)))
            oh, doh, l = o[b:e, h].double(), do[b:e, h].double(), lse[h, b:e, None].double()
            p = torch.exp(_logits(qh, kh, causal, scale) - l)
            delta = (doh * oh).sum(-1, keepdim=True)
            ds = p * (doh @ vh.T - delta)
            out["dv"][b:e, n] += p.T @ doh
            out["dq"][b:e, h] = scale * ds @ kh
            out["dk"][b:e, n] += scale * ds.T @ qh
            # P off by the logits' errors and LSE's product with log2 e; dP and delta sums of D products in fp32; P and
            # dS rounded to bf16, the products' sums in fp32
            slack = _slack(qh, kh, D, scale) * 2 + l.abs() * 8 * FP32
            sums = (D + 8) * 2 * FP32 * (doh.abs() @ vh.abs().T + (doh * oh).abs().sum(-1, keepdim=True))
            rest = 2.0 ** -18
            p_off = p * (BF16 * 1.01 + slack + rest)
            ds_off = ds.abs() * (BF16 * 1.01 + slack + rest) + p * sums
            tol["dv"][b:e, n] += p_off.T @ doh.abs()
            tol["dq"][b:e, h] = scale * ds_off @ kh.abs()
            tol["dk"][b:e, n] += scale * ds_off.T @ qh.abs()
    for n in out:
        tol[n] += BF16 * 1.01 * out[n].abs() + 1e-37
    return out, tol


def check(got, want, tol, what):
    """Every element within its bound (NaN is not)."""
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} elements, the first at {bad.nonzero()[0].tolist()}: " \
                          f"{float(off[bad][0])} over {float(tol[bad][0])}"
