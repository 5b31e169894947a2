"""Cases of attention over packed sequences and of rotary positions: what the operators compute, in
elementary torch operations, and the same calls through the library.

Packed: the tokens of several sequences of different lengths lie one behind the other, q [T, H, D], k and v
[T, Hkv, D], and `cu` (int32 [S + 1]) says where each begins and the last one ends.  Operators:

  prompt        attention of every sequence over itself (prompts, documents): O and LSE
  prompt_grad   its gradients dQ, dK, dV from dO, O and LSE
  rotary        queries and keys turned by the angles of their positions: for packed sequences, and for the
                new tokens of a serving step
  rotary_grad   the gradients back through the turn
"""
import math
import random

import torch

own = False


def listed():
    a = dict(op="prompt", H=32, Hkv=8, D=128, causal=True, fused=False)
    g = dict(a, op="prompt_grad")
    r = dict(op="rotary", H=32, Hkv=8, D=128, rot=128, interleaved=False, scaling="none", factor=1.0, base=10000.0, far=0, packed=True, fused=False)
    return [
        # one user's short prompt: the time to its first token
        dict(a, name="prompt_short", S=1, lo=700, hi=700),
        # the prompts that a server takes in one step, q, k and v as one projection wrote them
        dict(a, name="prompt_batch", S=24, lo=17, hi=2048, fused=True),
        # one long prompt, a share of the heads
        dict(a, name="prompt_long", S=1, H=16, Hkv=2, lo=16001, hi=16001),
        # an encoder's inputs: not causal, heads of their own, D = 64
        dict(a, name="encoder_d64", S=10, H=24, Hkv=24, D=64, lo=333, hi=2500, causal=False),
        # a fine-tuning step on a few short examples
        dict(g, name="grad_short", S=4, H=16, Hkv=4, lo=50, hi=400),
        # documents of many lengths in one pretraining step
        dict(g, name="grad_docs", S=20, H=16, Hkv=16, lo=100, hi=2048, fused=True),
        # one long document
        dict(g, name="grad_long", S=1, H=32, Hkv=8, lo=8192, hi=8192),
        # the encoder's gradients
        dict(g, name="grad_d64", S=10, H=24, Hkv=24, D=64, lo=333, hi=2500, causal=False),
        # a decoding step: one token for each of many sequences, far from their beginnings, half of each head turned
        dict(r, name="turn_token", S=64, lo=1, hi=1, rot=64, interleaved=True, scaling="ramp", factor=8.0, far=100000, packed=False),
        # the documents of a training step, q and k as the projection wrote them
        dict(r, name="turn_docs", S=24, lo=100, hi=2048, fused=True),
        # a long prompt with a raised base, at a chunk's place far behind its beginning
        dict(r, name="turn_long", S=1, lo=32768, hi=32768, scaling="base", factor=16.0, far=900000, interleaved=True),
        # the documents' gradients
        dict(r, name="turn_grad", op="rotary_grad", S=24, lo=100, hi=2048),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(1, 16), (2, 8), (8, 4), (4, 4), (16, 1), (24, 1), (2, 7), (3, 5), (4, 3), (1, 1), (8, 2), (12, 2)]


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt_grad", "prompt_grad", "rotary", "rotary_grad"])
    Hkv, G = rng.choice(_HEADS)
    c = dict(op=op, H=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128]))
    S = _log(rng, 1, 64)
    if op.startswith("prompt"):
        # the padded logits of the plain form, and the work of the largest listed case, bound the lengths
        causal = rng.random() < 0.7
        pairs = min(3e9, 1e12 / (c["D"] * (4 if op == "prompt" else 10) * (0.5 if causal else 1.0)))
        hi = _log(rng, 1, min(16001, int(math.sqrt(pairs / (S * Hkv * G)))))
        return c | dict(S=S, causal=causal, fused=rng.random() < 0.4, lo=rng.choice([0, 1, hi // 9, hi]), hi=hi)
    rot = rng.choice([c["D"], c["D"], c["D"] // 2, 16, 48])
    scaling = rng.choice(["none", "linear", "base", "ramp"])
    hi = _log(rng, 1, max(1, 32768 * 40 // (S * Hkv * (G + 1))))
    return c | dict(S=S, lo=rng.choice([0, 1, hi // 3, hi]) if (packed := rng.random() < 0.6) else hi, hi=hi, rot=rot, packed=packed, fused=packed and rng.random() < 0.4,
                    interleaved=rng.random() < 0.5, scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 32.0]),
                    base=rng.choice([10000.0, 500000.0]), far=rng.choice([0, 0, 5000, 1000000]))


def _lengths(case, seed):
    """The sequences' lengths.  Another seed has the same ones in another order."""
    r = random.Random("%d %d %d" % (case["S"], case["lo"], case["hi"]))
    lens = [case["hi"]] + [int(round(math.exp(r.uniform(math.log(case["lo"] + 1), math.log(case["hi"] + 1))))) - 1 for _ in range(case["S"] - 1)]
    random.Random("order %d" % seed).shuffle(lens)
    return lens


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens = _lengths(case, seed)
    H, Hkv, D, S, T = case["H"], case["Hkv"], case["D"], case["S"], sum(lens)
    s = {n: case[n] for n in ("op", "H", "Hkv", "D")}

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(device="cuda", dtype=torch.int32)
    if case["op"].startswith("prompt"):
        q, k, v = normal(T, H, D), normal(T, Hkv, D), normal(T, Hkv, D)
        k = k + 2.0 * normal(1, Hkv, D) * (torch.rand((1, Hkv, D), device="cuda", generator=gen) < 0.05)   # channels with a mean of their own
        x = torch.cat((q * 1.5, k, v), 1).to(torch.bfloat16)
        s |= dict(cu=cu, causal=case["causal"], longest=max(lens))
        s["q"], s["k"], s["v"] = x.split((H, Hkv, Hkv), 1)
        if not case["fused"]:
            s |= {n: s[n].contiguous() for n in ("q", "k", "v")}
        if case["op"] == "prompt_grad":
            s["do"] = normal(T, H, D).to(torch.bfloat16)
            s["o"], s["lse"] = _forward(s)                                     # what the step's forward pass left
    else:
        far = case["far"]
        start = (torch.rand(S, device="cuda", generator=gen) * far).to(torch.int32) if far else None
        shape = (T, H, D) if case["packed"] else (S, H, lens[0], D)
        s |= {n: case[n] for n in ("rot", "interleaved", "base", "scaling", "factor")}
        s |= dict(cu=cu if case["packed"] else None, start=start)
        x = normal(*(H + 2 * Hkv if i == 1 else n for i, n in enumerate(shape))).to(torch.bfloat16)
        s["q"], s["k"] = x[:, :H], x[:, H:H + Hkv]
        if not case["fused"]:
            s |= {n: s[n].contiguous() for n in ("q", "k")}
    if own:
        import bit_trainable_attention_sagebwd_gb300 as sa
        if case["op"].startswith("prompt"):
            s["ws"] = sa.alloc_packed_ws(T, S, H, Hkv, D, backward=case["op"] == "prompt_grad")
        else:
            s["table"] = sa.rotary_table(s["rot"], base=s["base"], scaling=s["scaling"], factor=s["factor"], context=_CONTEXT, interleaved=s["interleaved"])
    return s


# ------------------------------------------------------------------- plain forms

_CONTEXT = 4096                # the length that a scaled model was trained at
_FAST, _SLOW = 32.0, 1.0       # turns over it: pairs with more keep their frequency, with fewer take it over the factor


def _padded(x, s):
    """x [T, heads, D] as fp32 [S, Hkv, heads / Hkv, longest, D], zeros behind each sequence."""
    cu = s["cu"].long()
    at = cu[:-1, None] + torch.arange(s["longest"], device=x.device)
    live = at < cu[1:, None]
    x = x[at.clamp(max=x.shape[0] - 1)].float() * live[:, :, None, None]
    return x.unflatten(2, (s["Hkv"], -1)).permute(0, 2, 3, 1, 4)


def _packed(x, s):
    """_padded's inverse."""
    cu = s["cu"].long()
    live = torch.arange(s["longest"], device=x.device) < (cu[1:] - cu[:-1])[:, None]
    return x.permute(0, 3, 1, 2, 4).flatten(2, 3)[live]


def _seen(s):
    """Which keys each query sees [S, 1, 1, longest, longest] (causal: [.., 1] in the first place too)."""
    j = torch.arange(s["longest"], device=s["q"].device)
    seen = (j < (s["cu"][1:] - s["cu"][:-1])[:, None])[:, None, None, None, :]
    return seen & (j <= j[:, None]) if s["causal"] else seen


def _logits(s):
    t = (_padded(s["q"], s) / math.sqrt(s["D"])) @ _padded(s["k"], s).transpose(-1, -2)
    return t.masked_fill_(~_seen(s), -math.inf)


def _forward(s):
    if s["q"].shape[0] == 0:
        return torch.empty_like(s["q"]), s["q"].new_empty((s["H"], 0), dtype=torch.float32)
    t = _logits(s)
    m = t.amax(-1, keepdim=True).clamp(min=-1e30)                              # (a sequence of no tokens has no keys)
    p = t.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = _packed((p @ _padded(s["v"], s)) / l.clamp(min=1e-30), s).to(torch.bfloat16)
    return o, _packed(m + l.clamp(min=1e-30).log(), s)[:, :, 0].T.contiguous()


def _backward(s):
    if s["q"].shape[0] == 0:
        return tuple(torch.empty_like(s[n]) for n in ("q", "k", "v"))
    q, k, v, o, do = (_padded(s[n], s) for n in ("q", "k", "v", "o", "do"))
    lse = _padded(s["lse"].T[:, :, None], s)
    p = _logits(s).sub_(lse).exp_()
    dv = (p.transpose(-1, -2) @ do).sum(2, keepdim=True)
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).div_(math.sqrt(s["D"]))
    dq, dk = ds @ k, (ds.transpose(-1, -2) @ q).sum(2, keepdim=True)
    return tuple(_packed(x, s).to(torch.bfloat16) for x in (dq, dk, dv))


def _frequencies(s):
    """Radians a position of each pair, in 64 bits, and the factor of the turned channels."""
    rot, base, factor, scaling = s["rot"], s["base"], s["factor"], s["scaling"]
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    if scaling == "linear":
        f = f / factor
    if scaling != "ramp":
        return f, 1.0
    # between the pair that turns _FAST times over the context and the one that turns _SLOW times the share grows with its number
    first, last = (rot * math.log(_CONTEXT / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (_FAST, _SLOW))
    first, last = max(0, math.floor(first)), min(rot - 1, math.ceil(last))
    share = ((torch.arange(rot // 2, device="cuda", dtype=torch.float64) - first) / max(last - first, 1e-3)).clamp(0, 1)
    return f * (1 - share) + f / factor * share, 0.1 * math.log(factor) + 1.0


def _positions(s):
    """[T] or [S, N]."""
    if s["cu"] is None:
        at = torch.arange(s["q"].shape[2], device="cuda").expand(s["q"].shape[0], -1)
        return at if s["start"] is None else at + s["start"][:, None]
    cu = s["cu"].long()
    of = torch.repeat_interleave(torch.arange(cu.numel() - 1, device="cuda"), cu[1:] - cu[:-1], output_size=s["q"].shape[0])
    at = torch.arange(s["q"].shape[0], device="cuda") - cu[of]
    return at if s["start"] is None else at + s["start"][of]


def _turn(x, s, cos, sin):
    y, r = x.float(), s["rot"]
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if s["interleaved"] else (y[..., :r // 2], y[..., r // 2:r])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, w), -1).flatten(-2) if s["interleaved"] else torch.cat((u, w), -1)
    return torch.cat((turned, y[..., r:]), -1).to(x.dtype)


def _rotary(s):
    f, gain = _frequencies(s)
    angle = _positions(s).double()[..., None] * f
    angle = angle.unsqueeze(-2 if s["cu"] is not None else 1)                  # the same for every head
    cos, sin = (angle.cos() * gain).float(), (angle.sin() * gain).float()
    if s["op"] == "rotary_grad":
        sin = -sin
    return {"q": _turn(s["q"], s, cos, sin), "k": _turn(s["k"], s, cos, sin)}


def run(s):
    if own:
        import bit_trainable_attention_sagebwd_gb300 as sa
    if s["op"] == "prompt":
        o, lse = sa.packed_forward(s["q"], s["k"], s["v"], s["cu"], causal=s["causal"], ws=s["ws"]) if own else _forward(s)
        return {"o": o, "lse": lse}
    if s["op"] == "prompt_grad":
        if own:
            dq, dk, dv = sa.packed_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["cu"], causal=s["causal"], ws=s["ws"])
        else:
            dq, dk, dv = _backward(s)
        return {"dq": dq, "dk": dk, "dv": dv}
    if not own:
        return _rotary(s)
    turn = sa.rotary if s["op"] == "rotary" else sa.rotary_backward
    q, k = turn(s["table"], s["q"], s["k"], cu_seqlens=s["cu"], start=s["start"])
    return {"q": q, "k": k}


# ------------------------------------------------------------------- work, and 64 bits

def work(case):
    H, Hkv, D, lens = case["H"], case["Hkv"], case["D"], _lengths(case, 0)
    T = sum(lens)
    if case["op"].startswith("rotary"):
        return {"bytes": max(1.0, 4.0 * T * (H + Hkv) * D), "flops": 3.0 * T * (H + Hkv) * case["rot"]}
    pairs = sum(n * (n + 1) / 2.0 if case["causal"] else float(n) * n for n in lens)
    if case["op"] == "prompt":
        return {"bytes": max(1.0, T * (4.0 * (H + Hkv) * D + 4.0 * H)), "flops": 4.0 * D * H * pairs}
    return {"bytes": max(1.0, T * (8.0 * (H + Hkv) * D + 4.0 * H)), "flops": 10.0 * D * H * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rotary"):
        return _exact_rotary(s)
    H, G, scale = s["H"], s["H"] // s["Hkv"], s["D"] ** -0.5
    names = ("o", "lse") if case["op"] == "prompt" else ("dq", "dk", "dv")
    out = {n: torch.zeros((H, s["q"].shape[0]) if n == "lse" else s["k" if n in ("dk", "dv") else "q"].shape, dtype=torch.float64, device="cuda") for n in names}
    ends = s["cu"].tolist()
    for b, e in zip(ends, ends[1:]):
        for h in range(H if e > b else 0):
            q, k, v = s["q"][b:e, h].double(), s["k"][b:e, h // G].double(), s["v"][b:e, h // G].double()
            t = torch.einsum("id,jd->ij", q, k) * scale
            if s["causal"]:
                t.masked_fill_(torch.ones_like(t, dtype=torch.bool).triu(1), -math.inf)
            if case["op"] == "prompt":
                out["lse"][h, b:e] = torch.logsumexp(t, -1)
                out["o"][b:e, h] = torch.softmax(t, -1) @ v
                continue
            do, o = s["do"][b:e, h].double(), s["o"][b:e, h].double()
            p = torch.exp(t - s["lse"][h, b:e, None].double())
            out["dv"][b:e, h // G] += torch.einsum("ij,id->jd", p, do)
            w = p * (torch.einsum("id,jd->ij", do, v) - (do * o).sum(-1)[:, None]) * scale
            out["dq"][b:e, h] = torch.einsum("ij,jd->id", w, k)
            out["dk"][b:e, h // G] += torch.einsum("ij,id->jd", w, q)
    return out


def _exact_rotary(s):
    """Pairs as complex numbers."""
    r, base, factor = s["rot"], s["base"], s["factor"]
    pair = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    gain = 1.0
    if s["scaling"] == "base":
        base *= factor ** (r / (r - 2.0))
    speed = torch.exp(-2.0 * pair / r * math.log(base))
    if s["scaling"] == "linear":
        speed /= factor
    elif s["scaling"] == "ramp":
        gain = 1.0 + 0.1 * math.log(factor)
        at = [r / 2.0 * math.log(_CONTEXT / turns / (2.0 * math.pi)) / math.log(base) for turns in (_FAST, _SLOW)]
        at = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        slow = torch.clip((pair - at[0]) / max(at[1] - at[0], 1e-3), 0.0, 1.0)
        speed *= 1.0 - slow + slow / factor
    if s["cu"] is None:
        at = torch.arange(s["q"].shape[2], device="cuda").double() + torch.zeros((s["q"].shape[0], 1), device="cuda")
        at = (at if s["start"] is None else at + s["start"].double()[:, None])[:, None, :]
    else:
        at = torch.zeros(s["q"].shape[0], dtype=torch.float64, device="cuda")
        ends = s["cu"].tolist()
        for i, (b, e) in enumerate(zip(ends, ends[1:])):
            at[b:e] = torch.arange(e - b, device="cuda") + (0 if s["start"] is None else int(s["start"][i]))
        at = at[:, None]
    turn = torch.polar(torch.full_like(at, gain)[..., None].expand(*at.shape, r // 2).contiguous(), at[..., None] * speed)
    if s["op"] == "rotary_grad":
        turn = turn.conj()

    def turned(x):
        y = x.double().clone()
        a, b = (slice(0, r, 2), slice(1, r, 2)) if s["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        z = torch.complex(y[..., a], y[..., b]) * turn
        y[..., a], y[..., b] = z.real, z.imag
        return y

    return {"q": turned(s["q"]), "k": turned(s["k"])}
