"""The paged cache's calls in plain fp64 (and plain integers), request by request, for the tests.

Nothing here shares code with the library; tensors come and go as CPU torch tensors."""
from __future__ import annotations

import math
import random

import torch

F64 = torch.float64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step of a rounding, relative


def pages_of(n: int, page: int) -> int:
    return -(-n // page)


def extend(new, ctx, table, free, count, page, T):
    """think_extend_pages in plain integers: (kv_lens, table, count, q_start, positions, slots, some request refused)."""
    table = [list(r) for r in table]
    limit = len(table[0]) * page if table else 0
    lens, q_start, positions, slots = [], [0], [], []
    wanted, used, refused, row = 0, 0, False, 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        n, c = max(n, 0), max(c, 0)
        row += n
        need = pages_of(c + n, page) - pages_of(c, page)
        ok = c + n <= limit and row <= T
        if ok and need:
            wanted += need
            ok = wanted <= count
        if ok:
            for j in range(pages_of(c, page), pages_of(c + n, page)):
                table[b][j] = free[count - 1 - used]
                used += 1
        refused = refused or (not ok and n > 0)
        for i in range(n):
            p = c + i
            positions.append(p)
            slots.append(table[b][p // page] * page + p % page if ok and table[b][p // page] >= 0 else -1)
        lens.append(c + n if ok else c)
        q_start.append(min(row, T))
    pad = max(0, T - len(positions))
    return lens, table, count - used, q_start, (positions + [0] * pad)[:T], (slots + [-1] * pad)[:T], refused


def turned(x, weight, eps, inv_freq, neighbours, positions):
    """Norm and rotation of [T,H,d] rows in fp64, and the magnitude |x1| + |x2| behind each channel (for error bounds)."""
    x = x.to(F64)
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.to(F64)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    y, size = x.clone(), x.abs()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + rot // 2)
        angle = positions.to(F64) * inv_freq[i].to(F64)
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def attend(q, k_cache, v_cache, table, q_start, lens, window, scale):
    """Attention in fp64.  Returns (out, size, logit): size[t,h,c] = sum_j p_j |V_jc|, logit[t,h] = the largest
    scale * sum_c |q_c K_jc| over the keys that the row sees.  Rows outside every request stay NaN."""
    T, Hq, d = q.shape
    Hkv, page = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    out = torch.full((T, Hq, d), math.nan, dtype=F64)
    size, logit = torch.zeros_like(out), torch.zeros(T, Hq, dtype=F64)
    for b in range(len(lens)):
        r0, n, kv = q_start[b], q_start[b + 1] - q_start[b], lens[b]
        if n == 0:
            continue
        p_first = kv - n
        lo = max(0, p_first - window + 1) if window else 0  # older keys are seen by no row
        keys = list(range(lo, kv))
        if keys:
            where = torch.tensor([table[b][j // page] * page + j % page for j in keys])
            k = k_cache.transpose(1, 2).reshape(-1, Hkv, d)[where].to(F64)  # [keys, Hkv, d]
            v = v_cache.transpose(1, 2).reshape(-1, Hkv, d)[where].to(F64)
        j = torch.tensor(keys, dtype=torch.long)
        pos = p_first + torch.arange(n)
        seen = j[None] <= pos[:, None]
        if window:
            seen &= j[None] > pos[:, None] - window
        for h in range(Hq):
            rows = out[r0:r0 + n, h]
            rows.zero_()
            if not keys:
                continue
            qq = q[r0:r0 + n, h].to(F64)
            kk, vv = k[:, h // G], v[:, h // G]
            z = torch.where(seen, scale * (qq @ kk.T), -math.inf)
            top = z.max(-1, keepdim=True).values
            top = torch.where(top == -math.inf, 0.0, top)
            e = torch.exp(z - top)
            tot = e.sum(-1, keepdim=True)
            w = torch.where(tot > 0, e / tot, 0.0)
            rows.copy_(w @ vv)
            size[r0:r0 + n, h] = w @ vv.abs()
            logit[r0:r0 + n, h] = torch.where(seen, abs(scale) * (qq.abs() @ kk.abs().T), 0.0).max(-1).values
    return out, size, logit


def attend_bound(out, size, logit, dtype, keys: int):
    """How far the library's attention may be from `attend`, element by element.

    fp32 steps (unit u = 2^-24): a logit is a sum of 128 products in fp32, off by at most 128 u times the sum of their
    magnitudes (`logit`); the same holds where the products are formed from bf16 parts (fp32 tensors: 48 sums of 16
    products on the tensor core, each off by at most 2 u, and the parts' products that are left out, below 2 u: 98 u); a weight is the exponential of it (the argument's own rounding after the maximum is taken off:
    another 2 u |z| <= 2 u logit each for z and the maximum; the exponential itself to 2^-20), so its relative error is
    below r = 132 u logit + 2^-20.  Numerator and denominator each carry r, and sums over `keys` terms and as many
    rescalings add 2 keys u.  So |err| <= (2 r + 4 keys u) * size.
    bf16 inputs: the weights are rounded to bf16 for the product with V (half a step, 2^-8, of each term: 2^-8 size).
    The result is rounded to its type once: half a step of it."""
    u = 2.0 ** -24
    r = 132 * u * logit[..., None] + 2.0 ** -20
    err = (2 * r + 4 * keys * u) * size
    if dtype == torch.bfloat16:
        err = err + 2.0 ** -8 * size
    return err * (1 + 2.0 ** -6) + HALF_STEP[dtype] * out.abs() + 1e-30


class Batch:
    """Requests with random lengths, their pages in random order, garbage wherever no key is seen."""

    def __init__(self, new, ctx, Hq, Hkv, page, dtype, seed, window=0, layout="hnd", lens=None, poison=True, key_scale=1.0,
                 pad_rows=0):
        rng = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.new, self.page, self.window, self.dtype = list(new), page, window, dtype
        self.lens = [n + c for n, c in zip(new, ctx)] if lens is None else list(lens)
        B = len(new)
        self.q_start = [0]
        for n in new:
            self.q_start.append(self.q_start[-1] + n)
        self.T = self.q_start[-1] + pad_rows
        need = [pages_of(n, page) for n in self.lens]
        pool = sum(need) + 3
        order = list(range(pool))
        rng.shuffle(order)
        width = max(need + [1]) + 2
        self.table = [[-7] * width for _ in range(B)]
        shape = (pool, Hkv, page, 128)
        k = torch.randn(shape, generator=g) * key_scale
        v = torch.randn(shape, generator=g)
        if poison:
            live = torch.zeros(pool, page, dtype=torch.bool)
        for b in range(B):
            first_seen = max(0, self.lens[b] - new[b] - window + 1) // page if window else 0
            for j in range(need[b]):
                p = order.pop()
                if j >= first_seen:
                    self.table[b][j] = p
                    if poison:
                        live[p, :max(0, min(page, self.lens[b] - j * page))] = True
        if poison:  # rows that hold no key of a live page
            k.transpose(1, 2)[~live] = math.nan
            v.transpose(1, 2)[~live] = math.inf
        self.k, self.v = k.to(dtype), v.to(dtype)
        self.q = torch.randn((self.T, Hq, 128), generator=g).to(dtype)
        self.layout = layout

    def cache(self, x, device="cuda"):
        """The pool on the GPU, as [pages][head][row][d] or [pages][row][head][d] memory."""
        if self.layout == "nhd":
            return x.transpose(1, 2).contiguous().to(device).transpose(1, 2)
        return x.to(device)
