"""dQ where dS's rounding would be seen: keys with a large mean in common, which the true rows of dS cancel and their roundings do
not, and all of the weight on the keys whose roundings' rests go into dQ as well."""
import math

import torch

import packed_ref as ref

LENS = [17, 20, 32, 33, 50, 64, 65, 96, 97, 128, 130, 150, 200, 300]

# dQ's relative L2 error: its own rounding to bf16, uniform within half a step, is 2^-8 / sqrt 3 of a value at the most
# (0.0023; 0.0017 over all mantissas); the rests' own roundings, 2^-16 and five times that by the common mean, and fp32's do
# not show.  Without the rests it is 0.0054 to 0.0099, with their signs turned 0.010 and more, eight keys off 0.0028 to 0.0082.
MOST = 1.1 * 2.0 ** -8 / math.sqrt(3)


def carried(n):
    """Which of a sequence's keys have their rest carried: the first eight of every 32, in tiles of 128, as far as the
    tile's products go; of 32 keys or fewer the first sixteen."""
    at = torch.arange(n)
    place, keys = at % 128, torch.clamp(n - at // 128 * 128, max=128)
    return torch.where(keys <= 32, place < 16, (place % 32 < 8) & ((place < 64) | (keys > 96)))


def inputs(G, D, seed, device):
    """q, k, v, do, cu of sequences of LENS; one key/value head."""
    q, k, v, do, cu = ref.inputs(LENS, G, 1, D, seed=seed, device="cpu")
    k += 4.0
    q[:, :, 0] = 8.0
    k[:, 0, 0] = torch.cat([torch.where(carried(n), 2.0, -2.0) for n in LENS]).to(torch.bfloat16) * D ** 0.5   # logits 16, -16
    return [x.to(device) for x in (q, k, v, do, cu)]


def check(dq, want, cu):
    """Every sequence's error."""
    at = cu.tolist()
    for n, b, e in zip(LENS, at, at[1:]):
        off = float((dq[b:e].double() - want[b:e]).norm() / want[b:e].norm())
        assert off <= MOST, f"dQ of {n} tokens: relative L2 error {off}"
