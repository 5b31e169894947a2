"""Cases of the 8-bit paged key/value cache: what its operators compute, in elementary torch
operations, and the same calls through the library.

The cache of one layer is a pool of pages.  A page holds `page` tokens of every key/value head as
8-bit codes (int8 or e4m3) with one fp32 scale per (page, head) for K and one for V; a slot (one
sequence) lists its pages in a row of `table` and its number of tokens in `lengths`; `refs` counts
the slots that list a page (0: free).  Operators:

  append    quantizes new tokens into the pages their slot has reserved
  attention queries against the pages of their slot (one token, a few, or a chunk of a prompt)
  sample    fork, extend, truncate: several continuations share a prompt's pages, get room for
            their next tokens (a shared last page is copied first) and give their pages back
  compact   the live pages move to the front of another pool
"""
import math
import random

import torch

own = False

_TOP = {"int8": 127.0, "e4m3": 448.0}
_DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def listed():
    a = dict(op="attention", H=32, Hkv=8, D=128, page=64, kind="int8", causal=True, ragged_q=False)
    return [
        # one user, a short context: the latency of a token
        dict(a, name="token_short", B=1, Nq=1, lo=700, hi=700),
        # an ordinary decoding step of a server, contexts of many lengths
        dict(a, name="token_batch", B=64, Nq=1, lo=500, hi=8192),
        # a few long contexts (pages of 128 tokens, e4m3)
        dict(a, name="token_long", B=4, Nq=1, lo=100001, hi=131071, page=128, kind="e4m3"),
        # heads of their own, D = 64, not causal: tokens of a decoder against an encoder's states
        dict(a, name="cross_d64", B=12, H=24, Hkv=24, D=64, Nq=1, lo=333, hi=16384, page=32, kind="e4m3", causal=False),
        # drafted tokens to be verified, between one and four for each sequence
        dict(a, name="draft", B=16, Nq=4, lo=900, hi=16384, ragged_q=True),
        # a chunk of a long prompt behind what the cache holds of it
        dict(a, name="chunk", B=1, Nq=2048, lo=32768, hi=32768, kind="e4m3"),
        # the write of a decoding step: one token for each sequence, anywhere in its page
        dict(op="append", name="write_token", B=64, Hkv=8, D=128, page=64, kind="int8", lo=1, hi=1, start=4000, shift=True),
        # the write of two prompts of unlike lengths, the pages begun before
        dict(op="append", name="write_prompt", B=2, Hkv=8, D=128, page=64, kind="e4m3", lo=20001, hi=32768, start=100, shift=False),
        # four continuations of each of a few short prompts
        dict(op="sample", name="sample_few", B=4, n=4, Hkv=8, D=128, page=64, kind="int8", lo=100, hi=1500, room=1, spare=32),
        # eight continuations of each of many prompts, with room for a drafted run of tokens
        dict(op="sample", name="sample_many", B=32, n=8, Hkv=8, D=128, page=64, kind="int8", lo=1000, hi=8192, room=70, spare=2048),
        # a small pool, a third of it live
        dict(op="compact", name="compact_small", B=8, Hkv=4, D=64, page=16, kind="int8", lo=100, hi=1000, live=0.33),
        # a large pool, half of it live
        dict(op="compact", name="compact_large", B=32, Hkv=8, D=128, page=64, kind="e4m3", lo=8192, hi=32768, live=0.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "sample", "compact"])
    Hkv, G = rng.choice([(1, 32), (2, 4), (4, 4), (8, 4), (8, 1), (8, 2), (3, 5), (16, 1), (24, 1), (4, 8), (1, 1)])
    c = dict(op=op, Hkv=Hkv, D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), kind=rng.choice(["int8", "e4m3"]))
    if op == "attention":
        what = rng.choice(["one", "one", "few", "chunk"])
        c |= dict(H=Hkv * G, causal=rng.random() < 0.75, ragged_q=what != "one" and rng.random() < 0.6)
        if what == "chunk":
            Nq = _log(rng, 17, 2048)
            hi = _log(rng, Nq, 32768)
            return c | dict(B=rng.choice([1, 1, 2]) if Nq * hi * Hkv * G < (1 << 29) else 1, Nq=Nq, lo=max(0, hi - rng.randrange(0, 2000)), hi=hi)
        B = _log(rng, 1, 96)
        hi = _log(rng, 1, max(2, min(131071, (1 << 29) // (B * Hkv * c["D"]))))
        return c | dict(B=B, Nq=1 if what == "one" else rng.randrange(2, 17), lo=rng.choice([0, 1, hi // 10, hi]), hi=hi)
    if op == "append":
        B = _log(rng, 1, 64)
        hi = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, min(65536, (1 << 26) // (Hkv * c["D"])) // B))
        return c | dict(B=B, lo=rng.choice([0, 1, hi]), hi=hi, start=rng.choice([0, 17, 300, 5000]), shift=rng.random() < 0.5)
    if op == "sample":
        B = _log(rng, 1, 32)
        hi = _log(rng, 1, min(8192, (1 << 28) // (B * Hkv * c["D"])))
        return c | dict(B=B, n=rng.randrange(1, 9), lo=rng.choice([0, 1, hi // 3, hi]), hi=hi, room=rng.choice([1, 1, 4, 33, 70]), spare=_log(rng, 1, 2000))
    B, live = _log(rng, 1, 32), rng.uniform(0.1, 0.95)
    hi = _log(rng, 1, min(32768, int(live * (1 << 30)) // (B * Hkv * c["D"])))
    return c | dict(B=B, lo=rng.choice([0, hi // 4]), hi=hi, live=live)


def _pages(n, page):
    return -(-n // page)


def _lengths(case, seed, count):
    """Pairs of a sequence's start and length.  Another seed hands the same pairs to other
    sequences, so that the pool keeps its size."""
    r = random.Random("%s %d %d %d" % (case["op"], case["lo"], case["hi"], count))
    pairs = [(r.randint(0, case.get("start", 0)), r.randint(case["lo"], case["hi"])) for _ in range(count)]
    random.Random("order %d" % seed).shuffle(pairs)
    return [p for p, _ in pairs], [n for _, n in pairs]


def _quantized(x, kind):
    """Codes and scales of whole pages x [n_pages, Hkv, P, D]."""
    s = x.abs().amax(dim=(2, 3)) / _TOP[kind]
    return _codes(x, s[:, :, None, None], kind), s


def _codes(x, s, kind):
    """The codes of x under the scales s (0: code 0)."""
    q = torch.where(s > 0, x / s, torch.zeros_like(x))
    if kind == "int8":
        return q.round().clamp(-127.0, 127.0).to(torch.int8)
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _keys(shape, gen, gain):
    """Key-like values: some channels are far larger than the others."""
    return torch.randn(shape, device="cuda", generator=gen) * gain


def _new_cache(case, gen, lens, n_slots, reserved, extra, zeros=False):
    """A pool whose pages are strewn over it: slot i has `reserved[i]` pages, `extra` more are free.
    What no slot holds (free pages, the ends of last pages) keeps the codes of earlier use."""
    Hkv, D, page, kind = case["Hkv"], case["D"], case["page"], case["kind"]
    n_pages = sum(reserved) + extra
    max_pages = max(1, max(reserved) + 2 + _pages(case.get("room", 0), page))
    order = torch.randperm(n_pages, device="cuda", generator=gen, dtype=torch.int64).to(torch.int32)
    table = torch.full((n_slots, max_pages), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(reserved):
        table[i, :n] = order[at:at + n]
        at += n
    refs[order[:at].long()] = 1
    c = dict(table=table, lengths=torch.tensor(lens + [0] * (n_slots - len(lens)), dtype=torch.int32, device="cuda"), refs=refs,
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    gain = torch.exp(0.4 * torch.randn((1, Hkv, 1, D), device="cuda", generator=gen))
    for name, g in (("k", gain), ("v", torch.ones_like(gain))):
        if zeros:
            c[name] = torch.zeros((n_pages, Hkv, page, D), device="cuda").to(_DTYPE[kind])
            c[name + "_scale"] = torch.zeros((n_pages, Hkv), device="cuda")
        else:
            c[name], c[name + "_scale"] = _quantized(_keys((n_pages, Hkv, page, D), gen, g), kind)
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, Hkv, D, page, B = case["op"], case["Hkv"], case["D"], case["page"], case["B"]
    r = random.Random("slots %d" % seed)
    if op == "attention":
        _, lens = _lengths(case, seed, B)
        s = _new_cache(case, gen, lens, B, [_pages(n, page) for n in lens], 3)
        Nq = case["Nq"]
        s["q"] = (1.5 * torch.randn((B, case["H"], Nq, D), device="cuda", generator=gen)).to(torch.bfloat16)
        order = list(range(B))
        r.shuffle(order)
        s["slots"] = torch.tensor(order, dtype=torch.int32, device="cuda")
        s["q_len"] = torch.tensor([r.randint(1, Nq) for _ in range(B)], dtype=torch.int32, device="cuda") if case["ragged_q"] else None
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((B, case["H"], Nq), device="cuda")
    elif op == "append":
        pos, n_new = _lengths(case, seed, B)
        s = _new_cache(case, gen, [p + n for p, n in zip(pos, n_new)], B, [_pages(p + n, page) for p, n in zip(pos, n_new)], 3)
        gain = torch.exp(0.4 * torch.randn((1, Hkv, 1, D), device="cuda", generator=gen))
        shift = torch.randn((Hkv, D), device="cuda", generator=gen) if case["shift"] else None
        s["k_new"] = (_keys((B, Hkv, case["hi"], D), gen, gain) + (shift[None, :, None, :] if case["shift"] else 0.0)).to(torch.bfloat16)
        s["v_new"] = _keys((B, Hkv, case["hi"], D), gen, 1.0).to(torch.bfloat16)
        s["shift"] = shift
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
        s["n_new"] = torch.tensor(n_new, dtype=torch.int32, device="cuda")
    elif op == "sample":
        n, S = case["n"], B * (1 + case["n"])
        _, lens = _lengths(case, seed, B)
        s = _new_cache(case, gen, lens, S, [_pages(k, page) for k in lens], B * n * (1 + _pages(case["room"], page)) + case["spare"])
        s["src"] = torch.tensor([-1] * B + [i // n for i in range(B * n)], dtype=torch.int32, device="cuda")
        s["n_new"] = torch.tensor([0] * B + [case["room"]] * (B * n), dtype=torch.int32, device="cuda")
        s["keep"] = torch.tensor([-1] * B + [0] * (B * n), dtype=torch.int32, device="cuda")
        s["pos"] = torch.zeros(S, dtype=torch.int32, device="cuda")
        s["cow"] = torch.zeros(S, dtype=torch.int32, device="cuda")
    else:
        _, lens = _lengths(case, seed, B)
        need = [_pages(n, page) for n in lens]
        s = _new_cache(case, gen, lens, B, need, int(sum(need) * (1.0 / case["live"] - 1.0)) + 1)
        # as a fork leaves it: every fourth sequence begins with the first page of another
        for i in range(3, B, 4):
            if need[i] and need[0]:
                s["refs"][s["table"][i, 0].long()] -= 1
                s["table"][i, 0] = s["table"][0, 0]
                s["refs"][s["table"][0, 0].long()] += 1
        o = _new_cache(dict(case), gen, [0] * B, B, [0] * B, sum(need) + 1, zeros=True)
        o["table"] = torch.full_like(s["table"], -1)
        s["to"] = o
    s["page"], s["kind"], s["op"] = page, case["kind"], op
    s["causal"] = case.get("causal")
    if own:
        # the handle, and the workspace of the attention, that a serving program keeps
        import bit_trainable_attention_sagebwd_gb300 as sa
        s["cache"] = sa.KVCache(**{n: s[n] for n in _STATE})
        if op == "attention":
            s["ws"] = sa.alloc_kv_ws(s["cache"], B, case["H"], case["Nq"])
        if op == "compact":
            s["to_cache"] = sa.KVCache(**{n: s["to"][n] for n in _STATE})
            s["ws"] = sa.alloc_kv_compact_ws(s["cache"])
    return s


_STATE = ("k", "v", "k_scale", "v_scale", "table", "lengths", "refs", "status")


# ------------------------------------------------------------------- plain forms

def _attention(s):
    q, page = s["q"].float(), s["page"]
    B, H, Nq, D = q.shape
    Hkv = s["k"].shape[1]
    length = s["lengths"][s["slots"].long()].long()
    table = s["table"][s["slots"].long()].clamp(min=0).long()               # [B, M]
    S = table.shape[1] * page
    k = s["k"][table].float() * s["k_scale"][table][..., None, None]        # [B, M, Hkv, P, D]
    k = k.transpose(1, 2).reshape(B, Hkv, 1, S, D)
    v = s["v"][table].float() * s["v_scale"][table][..., None, None]
    v = v.transpose(1, 2).reshape(B, Hkv, 1, S, D)
    q_len = s["q_len"].long() if s["q_len"] is not None else torch.full_like(length, Nq)
    i, j = torch.arange(Nq, device=q.device), torch.arange(S, device=q.device)
    end = (length - q_len)[:, None] + i + 1 if s["causal"] else length[:, None].expand(B, Nq)
    seen = j < torch.minimum(end, length[:, None])[..., None]               # [B, Nq, S]
    t = torch.matmul(q.reshape(B, Hkv, H // Hkv, Nq, D), k.transpose(-1, -2)) / math.sqrt(D)
    t = t.masked_fill(~seen[:, None, None], -math.inf)
    m = t.amax(-1, keepdim=True)
    p = torch.exp(t - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.masked_fill(~(j < length[:, None])[:, None, None, :, None], 0.0)) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l))[..., 0]
    row = (i < q_len[:, None])[:, None, :]                                  # rows behind q_len stay as they were
    s["o"].copy_(torch.where(row[..., None], o.reshape(B, H, Nq, D), s["o"].float()))
    s["lse"].copy_(torch.where(row, lse.reshape(B, H, Nq), s["lse"]))
    return {"o": s["o"], "lse": s["lse"]}


def _append_one(s, pool, scale, x):
    """The pages that the new tokens touch, taken out, changed and put back."""
    page, kind = s["page"], s["kind"]
    B, Hkv, N, D = x.shape
    first = s["pos"].long() // page
    M = (N + page - 2) // page + 1                                           # pages that N tokens can touch
    j = first[:, None] + torch.arange(M, device=x.device)                    # [B, M] places in the table
    end = (s["pos"] + s["n_new"]).long()
    used = (s["n_new"] > 0)[:, None] & (j * page < end[:, None])
    ids = s["table"].gather(1, j.clamp(max=s["table"].shape[1] - 1)).clamp(min=0).long()
    token = j[..., None] * page + torch.arange(page, device=x.device)        # [B, M, P]
    new = (token >= s["pos"][:, None, None]) & (token < end[:, None, None])
    old = token < s["pos"][:, None, None]
    at = (token - s["pos"][:, None, None]).clamp(0, N - 1)
    fresh = x.gather(2, at.reshape(B, 1, M * page, 1).expand(B, Hkv, M * page, D)).reshape(B, Hkv, M, page, D).transpose(1, 2)
    was, codes = scale[ids], pool[ids].float()                               # [B, M, Hkv], [B, M, Hkv, P, D]
    new, old = new[:, :, None, :, None], old[:, :, None, :, None]
    top = torch.where(new, fresh.abs(), torch.zeros_like(fresh)).amax(dim=(3, 4)) / _TOP[kind]
    now = torch.where(old.any(3)[..., 0], torch.maximum(was, top), top)
    value = torch.where(new, fresh, codes * was[..., None, None])
    got = _codes(value, now[..., None, None], kind)
    same = ~new & (~old | (now == was)[..., None, None])                     # left as they were
    bits = torch.where(same, pool[ids].view(torch.int8), got.view(torch.int8))
    pool.view(torch.int8)[ids[used]] = bits[used]
    scale[ids[used]] = now[used]


def _append(s):
    k = s["k_new"].float()
    _append_one(s, s["k"], s["k_scale"], k - s["shift"][None, :, None, :] if s["shift"] is not None else k)
    _append_one(s, s["v"], s["v_scale"], s["v_new"].float())
    return {n: s[n] for n in ("k", "v", "k_scale", "v_scale")}


def _fork(s):
    page, table, lengths, src = s["page"], s["table"], s["lengths"], s["src"]
    to = src >= 0
    of = src.clamp(min=0).long()
    n = torch.where(to, lengths[of], torch.zeros_like(src))
    held = torch.arange(table.shape[1], device=table.device) < ((n + page - 1) // page)[:, None]
    rows = table[of]
    table.copy_(torch.where(held, rows, table))
    s["refs"] += torch.bincount(rows[held].long(), minlength=s["refs"].numel()).int()
    lengths.copy_(torch.where(to, n, lengths))


def _extend(s):
    page, table, lengths, refs, n = s["page"], s["table"], s["lengths"], s["refs"], s["n_new"]
    have, want = (lengths + page - 1) // page, (lengths + n + page - 1) // page
    last = table.gather(1, (have - 1).clamp(min=0).long()[:, None])[:, 0].clamp(min=0).long()
    copied = (n > 0) & (lengths % page > 0) & (refs[last] > 1)
    need = want - have + copied
    upto = need.cumsum(0)
    free = torch.nonzero(refs == 0)[:, 0].int()
    ok = (need == 0) | (upto <= free.numel())
    j = torch.arange(table.shape[1], device=table.device)
    begin = (have - copied.int())[:, None]
    taken = ok[:, None] & (j >= begin) & (j < want[:, None])
    rank = (upto - need)[:, None] + j - begin
    ids = torch.cat((free, free.new_zeros(1)))[rank.clamp(0, free.numel()).long()]
    table.copy_(torch.where(taken, ids, table))
    copied = copied & ok
    to = table.gather(1, (have - 1).clamp(min=0).long()[:, None])[:, 0].long()[copied]
    refs[ids[taken].long()] = 1
    refs -= torch.bincount(last[copied], minlength=refs.numel()).int()
    s["cow"].copy_(torch.where(copied, last.int(), torch.full_like(n, -1)))
    s["k"].view(torch.int8)[to] = s["k"].view(torch.int8)[last[copied]]
    s["v"].view(torch.int8)[to] = s["v"].view(torch.int8)[last[copied]]
    s["k_scale"][to] = s["k_scale"][last[copied]]
    s["v_scale"][to] = s["v_scale"][last[copied]]
    s["pos"].copy_(torch.where(ok, lengths, torch.full_like(n, -1)))
    lengths += torch.where(ok, n, torch.zeros_like(n))


def _truncate(s):
    page, table, lengths, keep = s["page"], s["table"], s["lengths"], s["keep"]
    now = torch.where(keep >= 0, torch.minimum(keep, lengths), lengths)
    j = torch.arange(table.shape[1], device=table.device)
    gone = (j >= ((now + page - 1) // page)[:, None]) & (j < ((lengths + page - 1) // page)[:, None])
    s["refs"] -= torch.bincount(table[gone].long(), minlength=s["refs"].numel()).int()
    lengths.copy_(now)


def _compact(s):
    o, page = s["to"], s["page"]
    live = torch.nonzero(s["refs"] > 0)[:, 0]
    n = live.numel()
    o["k"].view(torch.int8)[:n] = s["k"].view(torch.int8)[live]
    o["v"].view(torch.int8)[:n] = s["v"].view(torch.int8)[live]
    o["k_scale"][:n] = s["k_scale"][live]
    o["v_scale"][:n] = s["v_scale"][live]
    o["refs"].zero_()
    o["refs"][:n] = s["refs"][live]
    number = torch.cumsum(s["refs"] > 0, 0).int() - 1
    held = torch.arange(s["table"].shape[1], device=live.device) < ((s["lengths"] + page - 1) // page)[:, None]
    o["table"].copy_(torch.where(held, number[s["table"].clamp(min=0).long()], o["table"]))
    o["lengths"].copy_(s["lengths"])


def run(s):
    if own:
        import bit_trainable_attention_sagebwd_gb300 as sa
    if s["op"] == "attention":
        if not own:
            return _attention(s)
        o, lse = sa.kv_attention(s["q"], s["cache"], causal=s["causal"], slots=s["slots"], q_len=s["q_len"], o=s["o"], lse=s["lse"], ws=s["ws"])
        return {"o": o, "lse": lse}
    if s["op"] == "append":
        if not own:
            return _append(s)
        sa.kv_append(s["cache"], s["k_new"], s["v_new"], s["pos"], s["n_new"], k_shift=s["shift"])
        return {n: s[n] for n in ("k", "v", "k_scale", "v_scale")}
    if s["op"] == "sample":
        if own:
            sa.kv_fork(s["cache"], s["src"])
            sa.kv_extend(s["cache"], s["n_new"], pos=s["pos"], cow=s["cow"])
            sa.kv_truncate(s["cache"], s["keep"])
        else:
            _fork(s)
            _extend(s)
            _truncate(s)
        return {n: s[n] for n in ("k", "v", "k_scale", "v_scale", "table", "lengths", "refs", "pos", "cow")}
    if own:
        sa.kv_compact(s["cache"], s["to_cache"], ws=s["ws"])
    else:
        _compact(s)
    return {n: s["to"][n] for n in ("k", "v", "k_scale", "v_scale", "table", "lengths", "refs")}


# ------------------------------------------------------------------- work, and 64 bits

def work(case):
    """Bytes and operations of one pass with sequences of the mean length."""
    op, Hkv, D, page, B = case["op"], case["Hkv"], case["D"], case["page"], case["B"]
    mean = (case["lo"] + case["hi"]) / 2.0
    token = 2.0 * Hkv * (D + 4.0 / page)                                     # bytes of a cached token, its share of the scales included
    if op == "attention":
        H = case["H"]
        Nq = (case["Nq"] + 1) / 2.0 if case["ragged_q"] else case["Nq"]
        seen = max(0.0, mean - (Nq - 1) / 2.0) if case["causal"] else mean
        return {"bytes": B * mean * token + B * H * Nq * (4.0 * D + 4.0), "flops": max(1.0, 4.0 * B * H * Nq * seen * D)}
    if op == "append":
        return {"bytes": max(1.0, B * mean * (2.0 * Hkv * D * 2 + token)), "flops": 0.0}
    if op == "sample":
        # a copied page is read and written; the tables of the prompts are read and written n times, refs read once
        rows = B * case["n"]
        pages = math.ceil(mean / page)
        return {"bytes": rows * 2.0 * page * token + rows * pages * 8.0 + (B * pages + rows + case["spare"]) * 4.0, "flops": 0.0}
    pages = B * math.ceil(mean / page)
    return {"bytes": max(1.0, pages * (2.0 * page * token + 16.0)), "flops": 0.0}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s, case)
    if case["op"] == "append":
        return {"k": None, "v": None, "k_scale": _exact_scale(s, case, s["k_scale"], s["k_new"], s["shift"]), "v_scale": _exact_scale(s, case, s["v_scale"], s["v_new"], None)}
    return None                                                              # pages and numbers that only move


def _exact_attention(s, case):
    page, H, Hkv, D, Nq = case["page"], case["H"], case["Hkv"], case["D"], case["Nq"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    slots, table, lengths = s["slots"].tolist(), s["table"], s["lengths"].tolist()
    q_len = s["q_len"].tolist() if s["q_len"] is not None else [Nq] * len(slots)
    for b, slot in enumerate(slots):
        n, nq = lengths[slot], q_len[b]
        lse[b, :, :nq] = -math.inf
        ids = table[slot, :_pages(n, page)].long()
        for h in range(H if n else 0):
            hk = h // (H // Hkv)
            k = (s["k"][ids, hk].double() * s["k_scale"][ids, hk].double()[:, None, None]).reshape(-1, D)[:n]
            v = (s["v"][ids, hk].double() * s["v_scale"][ids, hk].double()[:, None, None]).reshape(-1, D)[:n]
            t = s["q"][b, h, :nq].double() @ k.T / math.sqrt(D)
            if case["causal"]:
                rows = torch.arange(nq, device="cuda")[:, None] + (n - nq)
                t = t.masked_fill(torch.arange(n, device="cuda")[None, :] > rows, -math.inf)
            lse[b, h, :nq] = torch.logsumexp(t, -1)
            o[b, h, :nq] = torch.nan_to_num(torch.softmax(t, -1)) @ v
    return {"o": o, "lse": lse}


def _exact_scale(s, case, scale, x, shift):
    page, top = case["page"], _TOP[case["kind"]]
    got = scale.double().clone()
    for b, (pos, n) in enumerate(zip(s["pos"].tolist(), s["n_new"].tolist())):
        new = x[b, :, :n].double()
        new = (new - shift.double()[:, None, :] if shift is not None else new).abs().amax(-1)      # [Hkv, n]
        for j in range(pos // page, _pages(pos + n, page) if n else 0):
            p = int(s["table"][b, j])
            most = new[:, max(0, j * page - pos):max(0, (j + 1) * page - pos)].amax(-1) / top
            got[p] = torch.maximum(got[p], most) if j * page < pos else most
    return got
