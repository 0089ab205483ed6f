"""The prompt side of the cache, measured: block tables and slot maps from request lengths, the per-head norm and
rotation with the write into the paged cache, attention of new tokens over the paged cache, and the gather of a
request's pages for the channel pruning.

A case is a dict of plain values.  The lengths of its requests follow from its own numbers (`mix` seeds them), so
that the work of a case is known without its inputs; the inputs follow from the seed given to `prepare`.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp32": 4}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a decode step's bookkeeping: 256 running requests, one new token each
        dict(name="pages: decode batch", op="pages", B=256, new_lo=1, new_hi=1, ctx_lo=16, ctx_hi=8192, page=16, mix=1),
        # the same for a batch of fresh and continued prompts, ragged
        dict(name="pages: ragged prompts", op="pages", B=33, new_lo=200, new_hi=4096, ctx_lo=0, ctx_hi=8192, page=64, mix=2),
        # one token of one request: the smallest call of a decode step
        dict(name="rope: one token", op="rope", T=1, Hkv=8, G=4, page=64, dtype="bf16", rot=128, pairs="halves",
             norm=True, far=131072),
        # a large prompt chunk, heads as in the grouped-query workloads
        dict(name="rope: 8192 tokens", op="rope", T=8192, Hkv=8, G=4, page=64, dtype="bf16", rot=128, pairs="halves",
             norm=True, far=131072),
        # fp32, odd row count, neighbouring pairs, partial rotation, no norm
        dict(name="rope: fp32 partial", op="rope", T=1777, Hkv=4, G=3, page=48, dtype="fp32", rot=96, pairs="neighbours",
             norm=False, far=32768),
        # decode of one request with a long context (the long-context workload's heads and length)
        dict(name="attn: long decode", op="attn", B=1, new_lo=1, new_hi=1, ctx_lo=131071, ctx_hi=131071, Hkv=8, G=4,
             page=64, window=0, dtype="bf16", mix=3),
        # a decode batch of ragged requests on small pages
        dict(name="attn: decode batch", op="attn", B=32, new_lo=1, new_hi=1, ctx_lo=500, ctx_hi=16000, Hkv=8, G=4,
             page=16, window=0, dtype="bf16", mix=4),
        # a whole prompt
        dict(name="attn: prompt 16384", op="attn", B=1, new_lo=16384, new_hi=16384, ctx_lo=0, ctx_hi=0, Hkv=8, G=4,
             page=64, window=0, dtype="bf16", mix=5),
        # chunked prompts beside running requests, with a sliding window and pages that do not divide a tile
        dict(name="attn: mixed window", op="attn", B=13, new_lo=1, new_hi=1500, ctx_lo=0, ctx_hi=12000, Hkv=4, G=8,
             page=48, window=4096, dtype="bf16", mix=6),
        # fp32, one query head a KV head
        dict(name="attn: fp32 chunks", op="attn", B=3, new_lo=90, new_hi=400, ctx_lo=0, ctx_hi=2500, Hkv=8, G=1,
             page=32, window=0, dtype="fp32", mix=7),
        # a long request handed to the channel pruning
        dict(name="gather: long request", op="gather", B=1, ctx_lo=131072, ctx_hi=131072, Hkv=8, page=64, dtype="bf16", mix=8),
        # a few short ragged ones in fp32
        dict(name="gather: ragged fp32", op="gather", B=5, ctx_lo=3, ctx_hi=1300, Hkv=4, page=48, dtype="fp32", mix=9),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    page = rng.choice([16, 16, 32, 48, 64, 64, 80, 128, 256])
    op = rng.choice(["pages", "rope", "rope", "attn", "attn", "attn", "attn", "gather"])
    mix = rng.randrange(1 << 30)
    if op == "pages":
        if rng.random() < 0.5:
            return dict(op=op, B=_log(rng, 1, 700), new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=_log(rng, 100, 30000), page=page, mix=mix)
        return dict(op=op, B=_log(rng, 1, 64), new_lo=1, new_hi=_log(rng, 2, 2000), ctx_lo=0, ctx_hi=_log(rng, 100, 30000),
                    page=page, mix=mix)
    if op == "rope":
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        return dict(op=op, T=_log(rng, 1, 8192 if dtype == "bf16" else 4096), Hkv=rng.choice([1, 2, 4, 8]),
                    G=rng.choice([1, 2, 3, 4, 4]), page=page, dtype=dtype, rot=rng.choice([128, 128, 64, 32, 96, 16]),
                    pairs=rng.choice(["halves", "neighbours"]), norm=rng.random() < 0.7, far=_log(rng, 10000, 500000), mix=mix)
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "gather":
        B = _log(rng, 1, 16)
        return dict(op=op, B=B, ctx_lo=1, ctx_hi=_log(rng, 1000, 131072 // B), Hkv=Hkv, page=page,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), mix=mix)
    kind = rng.choice(["decode", "decode", "prompt", "mixed", "mixed", "fp32"])
    window = rng.choice([0, 0, 0, _log(rng, 64, 8192)])
    if kind == "decode":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, new_lo=1, new_hi=rng.choice([1, 1, 1, 4]), ctx_lo=1, ctx_hi=_log(rng, 200, 131072 // B), Hkv=Hkv,
                    G=rng.choice([1, 2, 4, 4, 7, 8]), page=page, window=window, dtype="bf16", mix=mix)
    if kind == "prompt":
        n = _log(rng, 100, 12000)
        return dict(op=op, B=1, new_lo=n, new_hi=n, ctx_lo=0, ctx_hi=0, Hkv=Hkv, G=rng.choice([1, 2, 4]), page=page,
                    window=window, dtype="bf16", mix=mix)
    if kind == "mixed":
        return dict(op=op, B=_log(rng, 1, 12), new_lo=1, new_hi=_log(rng, 16, 1500), ctx_lo=0, ctx_hi=_log(rng, 100, 12000),
                    Hkv=Hkv, G=rng.choice([1, 2, 3, 4, 5]), page=page, window=window, dtype="bf16", mix=mix)
    return dict(op=op, B=_log(rng, 1, 8), new_lo=1, new_hi=_log(rng, 1, 400), ctx_lo=0, ctx_hi=_log(rng, 100, 4000), Hkv=Hkv,
                G=rng.choice([1, 2, 4]), page=page, window=window, dtype="fp32", mix=mix)


def _lengths(case):
    """New tokens and cached tokens of each request."""
    rng = random.Random(case["mix"])
    new, ctx = [], []
    for _ in range(case["B"]):
        new.append(_log(rng, case["new_lo"], case["new_hi"]) if "new_lo" in case else 0)
        ctx.append(rng.randint(case["ctx_lo"], case["ctx_hi"]))
    return new, ctx


def _pages(n, page):
    return -(-n // page)


def work(case):
    op = case["op"]
    if op == "pages":
        new, ctx = _lengths(case)
        fresh = sum(_pages(c + n, case["page"]) - _pages(c, case["page"]) for n, c in zip(new, ctx))
        # each page table entry that a slot needs, each fresh page read and written, lengths in and out, positions and slots
        return {"bytes": 12 * sum(new) + 8 * fresh + 16 * case["B"] + 12, "flops": sum(new)}
    e = _BYTES[case["dtype"]]
    if op == "rope":
        heads = case["Hkv"] * (case["G"] + 2)
        return {"bytes": case["T"] * (2 * heads * D * e + 12), "flops": case["T"] * heads * D * 6}
    new, ctx = _lengths(case)
    if op == "gather":
        return {"bytes": 2 * sum(ctx) * case["Hkv"] * D * e + 4 * sum(_pages(c, case["page"]) for c in ctx), "flops": 0}
    w = case["window"]
    pairs = keys = 0
    for n, c in zip(new, ctx):
        if w:
            first = max(0, c - w + 1)  # the oldest key that the first new token sees
            keys += c + n - first
            pairs += sum(min(c + i + 1, w) for i in range(n))
        else:
            keys += c + n
            pairs += n * c + n * (n + 1) // 2
    Hq = case["Hkv"] * case["G"]
    return {"bytes": 2 * keys * case["Hkv"] * D * e + 2 * sum(new) * Hq * D * e, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ inputs --

def _tables(case, lens, gen, dev):
    """A block table with the pages of `lens` tokens in a random order of the pool, -1 elsewhere, and the pool's size."""
    need = [_pages(n, case["page"]) for n in lens]
    total = sum(need)
    pool = total + max(2, total // 8)
    order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32, device=dev)
    rows = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(need)).to(dev)
    cols = torch.cat([torch.arange(n) for n in need]).to(dev)
    table[rows, cols] = order[:total]
    return table, order, total, pool


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, page = case["op"], case["page"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).to(dev)
    s = {"op": op, "page": page}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    if op == "pages":
        new, ctx = _lengths(case)
        # the running requests hold their pages; the table has room for the new ones, the free list is a stack of the rest
        need = [_pages(c, page) for c in ctx]
        after = [_pages(c + n, page) for n, c in zip(new, ctx)]
        table = torch.full((case["B"], max(after) + 3), -1, dtype=torch.int32, device=dev)
        order = torch.randperm(sum(after) + 9, generator=gen, device=dev).to(torch.int32)
        rows = torch.repeat_interleave(torch.arange(case["B"]), torch.tensor(need)).to(dev)
        cols = torch.cat([torch.arange(n) for n in need]).to(dev)
        table[rows, cols] = order[:sum(need)]
        T = sum(new)
        s.update(new=i32(new), ctx=i32(ctx), table=table, free=order[sum(need):].clone(), count=i32([sum(after) + 9 - sum(need)]),
                 lens_out=torch.zeros_like(i32(ctx)), count_out=i32([0]), q_start=i32([0] * (case["B"] + 1)),
                 positions=torch.zeros(T, dtype=torch.int32, device=dev), slots=torch.zeros(T, dtype=torch.int64, device=dev))
        return s
    dtype = _TYPES[case["dtype"]]
    Hkv, G = case["Hkv"], case.get("G", 1)
    if op == "rope":
        T = case["T"]
        heads = Hkv * (G + 2)
        # one projection's output: q, k and v heads beside each other in a row
        qkv = normal(T, heads, D).to(dtype)
        pool = _pages(T, page) + 2
        s.update(q=qkv[:, :Hkv * G], k=qkv[:, Hkv * G:Hkv * (G + 1)], v=qkv[:, Hkv * (G + 1):],
                 wq=(1 + 0.2 * normal(D)).to(dtype) if case["norm"] else None,
                 wk=(1 + 0.2 * normal(D)).to(dtype) if case["norm"] else None,
                 rot=case["rot"], pairs=case["pairs"], eps=1e-6,
                 freq=10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"]),
                 positions=torch.randint(0, case["far"], (1,), generator=gen, device=dev).to(torch.int32)
                 + torch.arange(T, dtype=torch.int32, device=dev),
                 slots=(torch.randperm(pool, generator=gen, device=dev)[:, None] * page
                        + torch.arange(page, device=dev)).reshape(-1)[:T].contiguous(),
                 k_cache=normal(pool, Hkv, page, D).to(dtype), v_cache=normal(pool, Hkv, page, D).to(dtype),
                 q_out=torch.zeros(T, Hkv * G, D, dtype=dtype, device=dev))
        return s
    new, ctx = _lengths(case)
    lens = [c + n for n, c in zip(new, ctx)]
    table, _, _, pool = _tables(case, lens, gen, dev)
    s.update(table=table, lens=i32(lens), host_lens=lens, host_new=new)
    k_cache = normal(pool, Hkv, page, D)
    # uneven channel magnitudes, as key caches have them
    k_cache *= torch.exp(0.5 * normal(Hkv, 1, D))
    s["k_cache"] = k_cache.to(dtype)
    if op == "gather":
        s["out"] = torch.zeros(case["B"], Hkv, max(lens), D, dtype=dtype, device=dev)
        return s
    T = sum(new)
    s.update(v_cache=normal(pool, Hkv, page, D).to(dtype), q=normal(T, Hkv * G, D).to(dtype),
             q_start=i32([0] + list(np.cumsum(new))), window=case["window"], scale=1.0 / math.sqrt(D),
             out=torch.zeros(T, Hkv * G, D, dtype=dtype, device=dev))
    return s


# ------------------------------------------------------------------ a pass --

_kept = {}


def _workspace(qdk, nbytes):
    """One workspace a size, zeroed once, as a serving program keeps it."""
    if nbytes not in _kept:
        _kept[nbytes] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    return _kept[nbytes]


def run(s):
    if own:
        import query_driven_key_b200 as qdk
        op = s["op"]
        if op == "pages":
            qdk.think_extend_pages(s["new"], s["ctx"], s["table"], s["free"], s["count"], s["page"], s["lens_out"],
                                   s["count_out"], s["q_start"], s["positions"], s["slots"],
                                   _workspace(qdk, qdk.think_extend_pages_workspace_size()))
            return s["lens_out"], s["count_out"], s["table"], s["q_start"], s["positions"], s["slots"]
        if op == "rope":
            qdk.think_norm_rope_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["eps"], s["freq"],
                                       s["pairs"] == "neighbours", s["positions"], s["slots"], s["q_out"], s["k_cache"],
                                       s["v_cache"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        if op == "attn":
            T, Hq, _ = s["q"].shape
            Hkv = s["k_cache"].shape[1]
            size = qdk.think_paged_attn_workspace_size(T, Hq, Hkv, dtype=s["q"].dtype)
            qdk.think_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["lens"], s["out"],
                                 _workspace(qdk, size), window=s["window"], scale=s["scale"], max_new=max(s["host_new"]))
            return s["out"]
        qdk.think_gather_pages(s["k_cache"], s["table"], s["lens"], s["out"])
        return s["out"]
    return _PLAIN[s["op"]](s)


def _plain_pages(s):
    new, ctx, page = s["new"].long(), s["ctx"].long(), s["page"]
    before, after = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    ends = torch.cumsum(after - before, 0)
    starts = ends - (after - before)
    q_start = torch.cat([torch.zeros_like(ends[:1]), torch.cumsum(new, 0)])
    # the k-th page handed out lies k below the top of the free stack
    col = torch.arange(s["table"].shape[1], device=new.device)[None]
    fresh = (col >= before[:, None]) & (col < after[:, None])
    k = starts[:, None] + col - before[:, None]
    at = torch.where(fresh, s["count"].long() - 1 - k, 0)
    s["table"].copy_(torch.where(fresh, s["free"][at], s["table"]))
    T = s["positions"].shape[0]
    row = torch.repeat_interleave(torch.arange(new.shape[0], device=new.device), new, output_size=T)
    pos = ctx[row] + torch.arange(T, device=new.device) - q_start[row]
    slots = s["table"][row, pos // page].long() * page + pos % page
    return ((ctx + new).int(), (s["count"] - ends[-1:]).int(), s["table"], q_start.int(), pos.int(), slots)


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["freq"][None]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        rot = s["rot"]
        if s["pairs"] == "halves":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([y, x[..., rot:]], -1)

    dtype, page = s["q"].dtype, s["page"]
    q = turned(s["q"], s["wq"]).to(dtype)
    p, i = s["slots"] // page, s["slots"] % page
    s["k_cache"][p, :, i] = turned(s["k"], s["wk"]).to(dtype)
    s["v_cache"][p, :, i] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _plain_attn(s):
    dev, page = s["q"].device, s["page"]
    T, Hq, _ = s["q"].shape
    B, Hkv = s["table"].shape[0], s["k_cache"].shape[1]
    G, M, N = Hq // Hkv, max(s["host_new"]), max(s["host_lens"])
    lens, first = s["lens"].long(), s["q_start"].long()[:-1]
    new = s["q_start"].long()[1:] - first
    cols = _pages(N, page)
    # keys and values of every request, padded to the longest: [B, Hkv, N, D]
    pages = s["table"][:, :cols].clamp(min=0).long()
    flat = lambda c: c[pages].transpose(1, 2).reshape(B, Hkv, cols * page, D)[:, :, :N].float()
    k, v = flat(s["k_cache"]), flat(s["v_cache"])
    j = torch.arange(N, device=dev)
    v = torch.where((j < lens[:, None])[:, None, :, None], v, 0.0)
    out = torch.zeros(T, Hq, D, dtype=s["q"].dtype, device=dev)
    step = max(1, min(M, (1 << 30) // (B * Hq * N)))  # rows at a time: the logits stay within a few GB
    for at in range(0, M, step):
        i = torch.arange(at, min(at + step, M), device=dev)
        real = i < new[:, None]
        rows = torch.where(real, first[:, None] + i, 0)
        q = s["q"][rows].float().reshape(B, len(i), Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, len(i) * G, D)
        z = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).view(B, Hkv, len(i), G, N)
        pos = (lens - new)[:, None, None] + i[None, :, None]
        seen = j <= pos
        if s["window"]:
            seen &= j > pos - s["window"]
        z.masked_fill_(~seen[:, None, :, None], -math.inf)
        top = z.amax(-1, keepdim=True)
        z = z.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
        total = z.sum(-1, keepdim=True)
        o = torch.matmul(z.view(B, Hkv, len(i) * G, N), v).view(B, Hkv, len(i), G, D)
        o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, len(i), Hq, D)
        out[rows[real]] = o[real].to(out.dtype)
    return out


def _plain_gather(s):
    B, Hkv, N, _ = s["out"].shape
    page = s["page"]
    cols = _pages(N, page)
    x = s["k_cache"][s["table"][:, :cols].clamp(min=0).long()].transpose(1, 2).reshape(B, Hkv, cols * page, D)[:, :, :N]
    keep = torch.arange(N, device=x.device) < s["lens"][:, None]
    return torch.where(keep[:, None, :, None], x, torch.zeros_like(x[:1, :1, :1, :1]))


_PLAIN = {"pages": _plain_pages, "rope": _plain_rope, "attn": _plain_attn, "gather": _plain_gather}


# ----------------------------------------------------------- in 64 bits --

def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "attn":
        return _exact_attn(s)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["host_lens"]):
        for c in range(_pages(n, s["page"])):
            at, m = c * s["page"], min(s["page"], n - c * s["page"])
            out[b, :, at:at + m] = s["k_cache"][int(s["table"][b, c]), :, :m].double()
    return out


def _exact_rope(s):
    """Each pair as a complex number times exp(i angle)."""
    turn = torch.polar(torch.ones_like(s["freq"])[None] * torch.ones(len(s["positions"]), 1, dtype=torch.float64, device="cuda"),
                       torch.outer(s["positions"].double(), s["freq"]))[:, None]
    half = s["rot"] // 2
    if s["pairs"] == "halves":
        re, im = torch.arange(half), torch.arange(half) + half
    else:
        re, im = torch.arange(half) * 2, torch.arange(half) * 2 + 1

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + s["eps"]) * w.double()
        y = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * turn
        x = x.clone()
        x[..., re], x[..., im] = y.real, y.imag
        return x

    page = s["page"]
    kc = s["k_cache"].double().transpose(1, 2).reshape(-1, *s["k_cache"].shape[1:2], D)
    vc = s["v_cache"].double().transpose(1, 2).reshape(-1, *s["k_cache"].shape[1:2], D)
    kc[s["slots"]] = one(s["k"], s["wk"])
    vc[s["slots"]] = s["v"].double()
    back = lambda c: c.reshape(-1, page, *c.shape[1:]).transpose(1, 2).contiguous()
    return one(s["q"], s["wq"]), back(kc), back(vc)


def _exact_attn(s):
    """Request by request and head by head."""
    T, Hq, _ = s["q"].shape
    G = Hq // s["k_cache"].shape[1]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, total) in enumerate(zip(s["host_new"], s["host_lens"])):
        pages = s["table"][b, :_pages(total, s["page"])].long()
        where = torch.arange(total, device="cuda")
        for h in range(s["k_cache"].shape[1]):
            k = s["k_cache"][pages, h].reshape(-1, D)[:total].double()
            v = s["v_cache"][pages, h].reshape(-1, D)[:total].double()
            for g in range(G):
                q = s["q"][row:row + n, h * G + g].double()
                z = (q @ k.t()) * s["scale"]
                back = (total - n + torch.arange(n, device="cuda"))[:, None] - where[None]  # how far behind the query a key lies
                hidden = (back < 0) | (back >= s["window"]) if s["window"] else back < 0
                z[hidden] = -math.inf
                out[row:row + n, h * G + g] = torch.softmax(z, -1) @ v
        row += n
    return out
