"""The paged cache in plain numpy, 64-bit where values are computed: what the tests compare with.
Pages, slots and tables are walked one at a time; fp32 roundings that the definition names are
made explicitly.  Imported by tests only."""
from __future__ import annotations

import numpy as np

TOP = {"int8": 127.0, "e4m3": 448.0}


def _e4m3_table():
    v = np.zeros(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        x = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v[b] = -x if b & 128 else x
    return v


E4M3 = _e4m3_table()  # (0x7f and 0xff, NaN in the format, are not written by the library)
_GRID = E4M3[:127]


def decode(b, kind):
    b = np.asarray(b, dtype=np.uint8)
    return b.view(np.int8).astype(np.float64) if kind == "int8" else E4M3[b]


def encode(x, kind):
    """x: fp32 quotients."""
    if kind == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(x.astype(np.float64)), 448.0)
    i = np.searchsorted(_GRID, a)
    lo, hi = np.maximum(i - 1, 0), np.minimum(i, 126)
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


class Cache:
    def __init__(self, n_pages, hkv, d, n_slots, max_pages, page, kind):
        self.page, self.kind = page, kind
        self.k = np.zeros((n_pages, hkv, page, d), np.uint8)
        self.v = np.zeros((n_pages, hkv, page, d), np.uint8)
        self.k_scale = np.zeros((n_pages, hkv), np.float32)
        self.v_scale = np.zeros((n_pages, hkv), np.float32)
        self.table = np.zeros((n_slots, max_pages), np.int32)
        self.lengths = np.zeros(n_slots, np.int32)
        self.refs = np.zeros(n_pages, np.int32)

    def pages(self, n):
        return -(-n // self.page)

    # ---- pages
    def fork(self, src):
        for s, f in enumerate(src):
            if f < 0:
                continue
            if f >= len(self.lengths) or src[f] >= 0 or self.lengths[s] != 0:
                continue
            n = self.pages(int(self.lengths[f]))
            self.table[s, :n] = self.table[f, :n]
            self.refs += np.bincount(self.table[f, :n], minlength=len(self.refs)).astype(np.int32)
            self.lengths[s] = self.lengths[f]

    def extend(self, n_new):
        S = len(self.lengths)
        pos, cow = np.full(S, -1), np.full(S, -1)
        free = [int(p) for p in np.flatnonzero(self.refs == 0)]
        refs0 = self.refs.copy()
        used, needed = 0, 0
        drop = []
        for s in range(S):
            n, length = int(n_new[s]), int(self.lengths[s])
            if n < 0 or length + n > self.table.shape[1] * self.page:
                continue
            have, want = self.pages(length), self.pages(length + n)
            shared = n > 0 and length % self.page and refs0[self.table[s, have - 1]] > 1
            need = want - have + bool(shared)
            needed += need
            if need and needed > len(free):
                continue
            take = free[needed - need:needed]
            used += need
            if shared:
                old, new = int(self.table[s, have - 1]), take.pop(0)
                cow[s] = old
                drop.append(old)
                self.table[s, have - 1] = new
                self.refs[new] = 1
                for a in (self.k, self.v, self.k_scale, self.v_scale):
                    a[new] = a[old]
            for i, p in enumerate(take):
                self.table[s, have + i] = p
                self.refs[p] = 1
            pos[s] = length
            self.lengths[s] += n
        for p in drop:
            self.refs[p] -= 1
        return pos.astype(np.int32), cow.astype(np.int32)

    def truncate(self, keep):
        for s, k in enumerate(keep):
            if k < 0:
                continue
            now = min(int(k), int(self.lengths[s]))
            for j in range(self.pages(now), self.pages(int(self.lengths[s]))):
                self.refs[self.table[s, j]] -= 1
            self.lengths[s] = now

    def compact(self, to):
        live = np.flatnonzero(self.refs > 0)
        if len(live) > len(to.refs):
            return False
        number = {int(p): i for i, p in enumerate(live)}
        for a, b in ((self.k, to.k), (self.v, to.v), (self.k_scale, to.k_scale), (self.v_scale, to.v_scale)):
            b[:len(live)] = a[live]
        to.refs[:] = 0
        to.refs[:len(live)] = self.refs[live]
        to.lengths[:] = self.lengths
        for s in range(len(self.lengths)):
            for j in range(self.pages(int(self.lengths[s]))):
                to.table[s, j] = number[int(self.table[s, j])]
        return True

    # ---- values
    def append(self, k, v, pos, n_new, slots=None, shift=None):
        """k, v: float32 values of the bf16 inputs [B, Hkv, Nn, D]."""
        for b in range(k.shape[0]):
            s = b if slots is None else int(slots[b])
            p0, n = int(pos[s]), int(n_new[s])
            if p0 < 0 or n <= 0:
                continue
            for x, codes, scale, sh in ((k, self.k, self.k_scale, shift), (v, self.v, self.v_scale, None)):
                for h in range(k.shape[1]):
                    new = x[b, h, :n].astype(np.float32)
                    if sh is not None:
                        new = new - sh[h].astype(np.float32)
                    for j in range(p0 // self.page, self.pages(p0 + n)):
                        page = self.table[s, j]
                        a, e = max(p0, j * self.page), min(p0 + n, (j + 1) * self.page)
                        part = new[a - p0:e - p0]
                        now = np.float32(np.abs(part).max()) * (np.float32(1) / np.float32(TOP[self.kind]))
                        off = a - j * self.page
                        if off:
                            was = scale[page, h]
                            now = max(now, was)
                            if now != was:
                                old = decode(codes[page, h, :off], self.kind).astype(np.float32) * was
                                codes[page, h, :off] = encode(old / now, self.kind)
                        codes[page, h, off:off + e - a] = encode(part / now, self.kind) if now > 0 else 0
                        scale[page, h] = now

    def values(self, s, h):
        """K and V of slot s, head h, in 64 bits: what its codes stand for."""
        n = int(self.lengths[s])
        ids = self.table[s, :self.pages(n)]
        d = self.k.shape[3]
        k = decode(self.k[ids, h], self.kind) * self.k_scale[ids, h].astype(np.float64)[:, None, None]
        v = decode(self.v[ids, h], self.kind) * self.v_scale[ids, h].astype(np.float64)[:, None, None]
        return k.reshape(-1, d)[:n], v.reshape(-1, d)[:n]

    def attention(self, q, causal=True, slots=None, q_len=None, sm_scale=None):
        """q: float64 [B, H, Nq, D].  Returns O, LSE and, for the tolerances, sum p |v| / l, sum |v| / l
        (l relative to the row's largest term), max_j sum_d |q k| scale and the mask of the rows that
        count."""
        B, H, Nq, D = q.shape
        hkv = self.k.shape[1]
        scale = 1.0 / np.sqrt(D) if sm_scale is None else sm_scale
        o, lse = np.zeros(q.shape), np.full((B, H, Nq), -np.inf)
        pv, av, mag = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, H, Nq))
        rows = np.zeros((B, H, Nq), bool)
        for b in range(B):
            s = b if slots is None else int(slots[b])
            n, nq = int(self.lengths[s]), Nq if q_len is None else int(q_len[b])
            rows[b, :, :nq] = True
            for h in range(H):
                k, v = self.values(s, h // (H // hkv))
                for i in range(nq):
                    end = min(n, max(0, n - nq + i + 1)) if causal else n
                    if end == 0:
                        continue
                    t = k[:end] @ q[b, h, i] * scale
                    m = t.max()
                    p = np.exp(t - m)
                    l = p.sum()
                    o[b, h, i] = p @ v[:end] / l
                    lse[b, h, i] = m + np.log(l)
                    pv[b, h, i] = p @ np.abs(v[:end]) / l
                    av[b, h, i] = np.abs(v[:end]).sum(0) / l
                    mag[b, h, i] = (np.abs(k[:end]) @ np.abs(q[b, h, i])).max() * scale
        return o, lse, pv, av, mag, rows


def attention_tolerances(o, lse, pv, av, mag, n, d):
    """How far O and LSE may be from the 64-bit values, from the roundings of the definition.

    S: fp32 products and sums of d exact terms, the scales and the exponent's argument: at most
    (d + 8) roundings of 2^-23 (a tensor core may truncate where fp32 rounds) of sum |q k|; each p,
    and with it l, is off by that factor and ex2's 2^-22, O twice (above and below the line).
    P in fp16: 2^-11 relative, 2^-25 absolute where it is subnormal.  Sums over n keys: n roundings
    of 2^-23 at most.  O in bf16: 2^-8."""
    ds = ((d + 8) * 2.0 ** -23) * mag + 2.0 ** -22 + n * 2.0 ** -23
    tol_o = (2.0 ** -11 + 2.2 * ds[..., None]) * pv + 2.0 ** -25 * av
    tol_o = tol_o + 2.0 ** -8 * (np.abs(o) + tol_o) + 1e-37
    return tol_o, ds + np.abs(lse) * 2.0 ** -22
