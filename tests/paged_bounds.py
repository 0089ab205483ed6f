"""What the attention over pages may be off by, closely enough that a lost piece of a long context or a lost part of an
fp32 number shows.  u = 2^-24, half a step of fp32.

paged_plain.attend_bound adds up the worst case of every sum over every key.  Over 100000 keys of either sign that is
more than the result.  Here the sums count as the kernels form them, and the rounding of the bf16 weights, whose errors
are independent of one another, counts with six times its standard deviation."""
from __future__ import annotations

import math

import torch

import paged_plain as P

F64 = torch.float64
U = 2.0 ** -24
PARTS = 148  # blocks that share the work


def exact(x: P.Batch, scale: float):
    """Attention of a Batch in fp64: out, size = sum p |V|, spread = sqrt(sum p^2 V^2), logit as in paged_plain.attend."""
    out, size, logit = P.attend(x.q, x.k, x.v, x.table, x.q_start, x.lens, x.window, scale)
    spread = torch.zeros_like(out)
    Hkv, G = x.k.shape[1], x.q.shape[1] // x.k.shape[1]
    for b, kv in enumerate(x.lens):
        r0, r1 = x.q_start[b], x.q_start[b + 1]
        if r0 == r1 or kv == 0:
            continue
        lo = max(0, kv - (r1 - r0) - x.window + 1) if x.window else 0
        j = torch.arange(lo, kv)
        at = torch.tensor(x.table[b])[j // x.page] * x.page + j % x.page
        back = (kv - (r1 - r0) + torch.arange(r1 - r0))[:, None] - j[None]
        seen = (back >= 0) & (back < x.window) if x.window else back >= 0
        for h in range(x.q.shape[1]):
            k = x.k.transpose(1, 2).reshape(-1, Hkv, 128)[at, h // G].to(F64)
            v = x.v.transpose(1, 2).reshape(-1, Hkv, 128)[at, h // G].to(F64)
            w = torch.softmax(torch.where(seen, scale * (x.q[r0:r1, h].to(F64) @ k.T), -1e300), -1)
            spread[r0:r1, h] = torch.sqrt((w * w) @ (v * v))
    return out, size, spread, logit


def chain(x: P.Batch, Hq: int, Hkv: int) -> int:
    """At most so many key tiles of an item are added up by one block: an equal share of all tiles, or an item of up to
    16 that is not cut, and one more at either border."""
    rows, keys = (256, 128) if x.dtype == torch.bfloat16 else (128, 64)
    total = 0
    for b, kv in enumerate(x.lens):
        n = x.q_start[b + 1] - x.q_start[b]
        seen = min(kv, n + x.window) if x.window else kv
        total += Hkv * -(-n * (Hq // Hkv) // rows) * (seen // keys + 6)  # (6: its cost and two borders)
    return total // PARTS + 18


def bound(out, size, spread, logit, dtype, tiles: int):
    """Weights: as in paged_plain.attend_bound, relative r = 132 u logit + 2^-20, in the numerator and in the sum.
    bf16: a tile's product adds 8 times to O, each off by at most 2 u of what is there (the tensor core drops what is
    below the last place); each weight's rounding to bf16 is off by at most 2^-8 of it, evenly spread at most, so
    that its standard deviation is below 2^-8 / sqrt(3).
    fp32: a tile's O is a sum of its own, whose 4 steps of the large terms are off by 2 u each and whose 20 of the small
    ones (2^-8 of it or less) by 2 u 2^-8 * 20 in all, below 9 u; it is added to the item's with half a step, u.
    Sum of the weights: 32 terms a lane and 3 joins of lanes, then one addition a tile: (35 + tiles) u.
    Joins: up to 2 partials of each part, with factors to 2^-21 and an addition of u each: (2 * 148 + 8) u and 2^-20."""
    r = 132 * U * logit[..., None] + 2.0 ** -20
    steps = (16 * tiles if dtype == torch.bfloat16 else 9 + tiles) + 35 + tiles + 2 * PARTS + 8
    err = (2 * r + steps * U + 2.0 ** -20) * size
    if dtype == torch.bfloat16:
        err = err + 6 * 2.0 ** -8 / math.sqrt(3.0) * spread
    return err * (1 + 2.0 ** -6) + P.HALF_STEP[dtype] * out.abs() + 1e-30


# new, ctx, Hq, Hkv, page, window
LONG = [([1], [150000], 4, 1, 64, 0), ([3], [120000], 8, 1, 16, 90001), ([200], [40000], 2, 1, 128, 0),
        ([1, 2, 1], [30000, 9, 60000], 8, 2, 32, 0)]


def long_batch(i: int, dtype) -> P.Batch:
    new, ctx, Hq, Hkv, page, window = LONG[i]
    return P.Batch(new, ctx, Hq, Hkv, page, dtype, 500 + i, window=window, layout="nhd" if i % 2 else "hnd", poison=False)


# ------------------------------------------- the three parts of an fp32 number --

def parts_of(x, n: int):
    """fp32 numbers as the sum of their first n bf16 parts, each the rounding of what the ones before it leave."""
    left, got = x.float().clone(), torch.zeros_like(x, dtype=F64)
    for _ in range(n):
        p = left.to(torch.bfloat16)
        got += p.to(F64)
        left = left - p.float()
    return got


def with_third_part(b):
    """bf16 numbers in [1, 2) -> fp32 numbers whose second part is 2^-9 and whose third is 0.45 * 2^-16."""
    return (b.double() + 2.0 ** -9 + 0.45 * 2.0 ** -16).float()


def two_key_case():
    """One token a request over two keys of which one channel is not 0, scale 1: with values 1 and -1 the output is
    tanh(z / 2), z = q k of the first key."""
    g = torch.Generator().manual_seed(3)
    near_one = lambda: (1 + torch.rand(64, generator=g) / 4).to(torch.bfloat16)
    q, k = with_third_part(near_one()), with_third_part(near_one())
    for x in (q, k):
        assert bool((parts_of(x, 3) == x.to(F64)).all()) and bool((x.to(F64) - parts_of(x, 2) > 0.4 * 2.0 ** -16).all())
    return q, k


def two_key_want(q, k):
    return torch.tanh(q.to(F64) * k.to(F64) / 2)


def two_key_bound(q, k):
    """z is one product of three parts each: terms left out below 3 u z, six sums that drop up to 2 u each, one product
    with the scale (u) and one sum (2 u): 18 u z, and d tanh(z / 2) is at most half of dz.  Two weights, each relative
    2^-22, move it by at most 2^-22 together; the argument's and the sums' roundings double that.  Sum and quotient 4 u."""
    return 9 * U * (q * k).to(F64) + 2.0 ** -21 + 4 * U


def mean_bound(tiles: int, logit: float = 0.0):
    """Weighted mean of positive values over `tiles` key tiles in one block, relative: 9 u in a tile; the tile sums grow
    about evenly, so their roundings have a standard deviation of at most u sqrt(tiles) / 3, counted six times, and so
    have those of the sum of the weights with its 35 u; the last product and quotient 3 u.  Weights that are not all
    exactly 1 add 2 r, r = 132 u logit + 2^-20 as in `bound`."""
    weights = 2 * (132 * U * logit + 2.0 ** -20) + (35 + 2 * math.sqrt(tiles)) * U if logit else 0.0
    return (9 + 2 * math.sqrt(tiles) + 3) * U + weights
