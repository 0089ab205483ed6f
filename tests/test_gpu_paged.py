"""The paged cache's kernels against plain fp64 and plain integers, on the GPU."""
import math
import random

import pytest
import torch

import paged_plain as P

pytestmark = pytest.mark.gpu
qdk = pytest.importorskip("query_driven_key_b200")

BF, F32 = torch.bfloat16, torch.float32
SCALE = 1.0 / math.sqrt(128.0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def ws(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def attn_ws(T, Hq, Hkv, dtype):
    """A workspace whose scratch holds NaN: only the status word and the counters have to be zero."""
    w = torch.full((qdk.think_paged_attn_workspace_size(T, Hq, Hkv, dtype=dtype),), 255, dtype=torch.uint8, device="cuda")
    w[:256 + 2048] = 0
    return w


# ------------------------------------------------------------- page tables --

def run_extend(new, ctx, table, free, count, page, T, in_place=False, n_free=None):
    B = len(new)
    lens, cnt = i32(ctx), i32([count])
    o = dict(new=i32(new), lens=lens, table=i32(table).reshape(B, -1), free=i32(free), cnt=cnt,
             lens_out=lens if in_place else i32([-5] * B), cnt_out=cnt if in_place else i32([-5]),
             q_start=i32([-5] * (B + 1)), pos=torch.full((T,), -5, dtype=torch.int32, device="cuda"),
             slots=torch.full((T,), -5, dtype=torch.int64, device="cuda"), ws=ws(qdk.think_extend_pages_workspace_size()))
    qdk.think_extend_pages(o["new"], o["lens"], o["table"], o["free"], o["cnt"], page, o["lens_out"], o["cnt_out"],
                           o["q_start"], o["pos"], o["slots"], o["ws"])
    return o


def check_extend(new, ctx, table, free, count, page, T, in_place=False):
    o = run_extend(new, ctx, table, free, count, page, T, in_place)
    lens, tab, left, q_start, pos, slots, refused = P.extend(new, ctx, table, free, count, page, T)
    assert o["lens_out"].tolist() == lens
    assert o["table"].tolist() == tab
    assert o["cnt_out"].item() == left
    assert o["q_start"].tolist() == q_start
    assert o["pos"].tolist() == pos
    assert o["slots"].tolist() == slots
    status = qdk.think_read_device_status(o["ws"])
    assert bool(status & qdk.THINK_DEVICE_NO_PAGES) == refused
    return status


def extend_case(B, hi_new, hi_ctx, page, seed, spare=5, width_extra=2):
    r = random.Random(seed)
    new = [r.randint(0, hi_new) for _ in range(B)]
    ctx = [r.randint(0, hi_ctx) for _ in range(B)]
    need = [P.pages_of(c, page) for c in ctx]
    fresh = sum(P.pages_of(c + n, page) for n, c in zip(new, ctx)) - sum(need)
    ids = list(range(sum(need) + fresh + spare))
    r.shuffle(ids)
    width = max(P.pages_of(c + n, page) for n, c in zip(new, ctx)) + width_extra
    table = [[ids.pop() for _ in range(k)] + [-1] * (width - k) for k in need]
    return new, ctx, table, ids, len(ids), page, sum(new)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,hi_new,hi_ctx,page", [
    (1, 1, 0, 16), (1, 0, 40, 16), (3, 70, 100, 48), (32, 1, 500, 16), (1024, 1, 90, 16), (1025, 3, 60, 16),
    (2100, 2, 40, 32), (7, 3000, 200, 64), (33, 1500, 4000, 256)])
def test_extend(B, hi_new, hi_ctx, page, in_place):
    status = check_extend(*extend_case(B, hi_new, hi_ctx, page, 11 * B + page), in_place=in_place)
    assert status == 0


@pytest.mark.parametrize("seed", range(4))
def test_extend_runs_out(seed):
    """Fewer free pages than wanted: the first requests are served, those that want none too."""
    new, ctx, table, free, count, page, T = extend_case(40, 90, 200, 32, 900 + seed, spare=0)
    for b in range(0, 40, 5):
        new[b], T = 0, T - new[b]
    for c in (0, 1, count // 3, count - 1):
        check_extend(new, ctx, table, free, c, page, T, in_place=bool(seed & 1))


def test_extend_no_room_in_table_or_rows():
    # request 1 outgrows its table row (4 pages of 16), request 3 the 50 rows
    check_extend([5, 30, 10, 20], [0, 40, 60, 0], [[-1] * 4, [1, 2, 3, -1], [4, 5, 6, 7], [-1] * 4], [8, 9, 10, 11], 4, 16, 50)
    # more rows than tokens: position 0 and slot -1 behind the last request; less than nothing counts as none
    check_extend([5, -3, 2], [0, 4, 17], [[-1] * 3, [0, -1, -1], [1, 2, -1]], [3, 4], 2, 16, 23)


def test_extend_bad_pages():
    status = check_extend([2, 20], [3, 5], [[-2, -1, -1], [4, -1, -1]], [7, -9, 5], 2, 16, 22)
    assert status == qdk.THINK_DEVICE_BAD_PAGE


def test_extend_count_above_stack_is_held_to_it():
    o = run_extend([16], [0], [[-1, -1]], [3, 6], 1000, 16, 16)
    assert o["table"].tolist() == [[6, -1]] and o["cnt_out"].item() == 1


# ----------------------------------------------------- norm, rotation, pages --

def rope_case(T, Hq, Hkv, dtype, rot, neighbours, norm, page, layout, seed, far=131072):
    g = torch.Generator().manual_seed(seed)
    heads = Hq + 2 * Hkv
    qkv = torch.randn((T, heads, 128), generator=g).to(dtype).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    wq, wk = ((1 + 0.3 * torch.randn((2, 128), generator=g)).to(dtype).cuda() if norm else (None, None))
    freq = None if rot == 0 else (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).cuda()
    pages = P.pages_of(T, page) + 2
    slots = torch.randperm(pages * page, generator=g)[:T]
    positions = torch.randint(0, far, (T,), generator=g).to(torch.int32)
    shape = (pages, Hkv, page, 128) if layout == "hnd" else (pages, page, Hkv, 128)
    caches = [torch.full(shape, 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    if layout == "nhd":
        caches = [c.transpose(1, 2) for c in caches]
    return q, k, v, wq, wk, freq, positions, slots, caches


@pytest.mark.parametrize("T,Hq,Hkv,dtype,rot,neighbours,norm,page,layout", [
    (1, 32, 8, BF, 128, False, True, 16, "hnd"), (1, 1, 1, F32, 128, True, True, 16, "hnd"),
    (37, 6, 2, BF, 96, False, True, 48, "nhd"), (37, 6, 2, BF, 96, True, False, 48, "nhd"),
    (130, 40, 40, BF, 64, False, False, 64, "hnd"), (19, 3, 1, F32, 16, False, True, 32, "nhd"),
    (64, 71, 3, F32, 128, False, True, 16, "hnd"), (5, 4, 2, BF, 0, False, True, 16, "hnd"),
    (9, 4, 2, F32, 0, True, False, 16, "hnd"), (11, 16, 1, BF, 32, True, True, 128, "hnd"),
    # several tokens a step (a block's tokens no multiple of them), and three head rows a thread group
    (2600, 1, 1, BF, 128, False, True, 64, "hnd"), (1301, 4, 2, F32, 128, True, True, 16, "nhd"), (603, 8, 4, BF, 64, True, True, 32, "hnd"),
    (600, 6, 1, F32, 96, False, True, 16, "hnd"), (310, 64, 8, BF, 128, False, True, 16, "hnd"), (19, 32, 8, F32, 128, True, True, 48, "nhd")])
def test_norm_rope_append(T, Hq, Hkv, dtype, rot, neighbours, norm, page, layout):
    eps = 1e-6
    q, k, v, wq, wk, freq, positions, slots, (kc, vc) = rope_case(T, Hq, Hkv, dtype, rot, neighbours, norm, page, layout, T + rot)
    bad = {3, 8} if T > 8 else set()
    for t, s in zip(sorted(bad), (-1, kc.shape[0] * page)):
        slots[t] = s
    q_out = torch.full((T, Hq, 128), 9.0, dtype=dtype, device="cuda")
    qdk.think_norm_rope_append(q, k, v, wq, wk, eps, freq, neighbours, positions.cuda(), slots.cuda(), q_out, kc, vc)
    cpu = lambda x: None if x is None else x.cpu()
    want_k = torch.full((kc.shape[0] * page, Hkv, 128), 7.0, dtype=P.F64)
    want_v, size_k = want_k.clone(), torch.zeros_like(want_k)
    yk, sk = P.turned(cpu(k), cpu(wk), eps, cpu(freq), neighbours, positions)
    for t in range(T):
        if t not in bad:
            want_k[slots[t]], size_k[slots[t]], want_v[slots[t]] = yk[t], sk[t], v[t].cpu().to(P.F64)
    flat = lambda c: c.cpu().transpose(1, 2).reshape(-1, Hkv, 128).to(P.F64)
    assert torch.equal(flat(vc), want_v)
    # fp32 steps (u = 2^-24): the mean square of 128 terms 128 u, its root half of that, rsqrt, two products 6 u;
    # cosine and sine to 8 u (argument and function); two products and a sum 3 u: below 90 u of |x1| + |x2|.
    # One rounding to the type.
    bound = lambda y, size: 90 * 2.0 ** -24 * size + P.HALF_STEP[dtype] * (1 + 2.0 ** -6) * y.abs() + 1e-30
    assert ((flat(kc) - want_k).abs() <= bound(want_k, size_k)).all()
    yq, sq = P.turned(cpu(q), cpu(wq), eps, cpu(freq), neighbours, positions)
    assert ((q_out.cpu().to(P.F64) - yq).abs() <= bound(yq, sq)).all()


def test_norm_rope_append_in_place_and_keys_only():
    q, k, v, wq, wk, freq, positions, slots, (kc, vc) = rope_case(50, 8, 2, BF, 128, False, True, 16, "hnd", 5)
    pos, sl = positions.cuda(), slots.cuda()
    out = torch.empty((50, 8, 128), dtype=BF, device="cuda")
    qdk.think_norm_rope_append(q, k, v, wq, wk, 1e-5, freq, False, pos, sl, out, kc, vc)
    kc2, vc2 = torch.full_like(kc, 7.0), torch.full_like(vc, 7.0)
    qdk.think_norm_rope_append(q[:, :0], k, v, None, wk, 1e-5, freq, False, pos, sl, out[:, :0], kc2, vc2)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)
    qdk.think_norm_rope_append(q, k, v, wq, wk, 1e-5, freq, False, pos, sl, q, kc2, vc2)
    assert torch.equal(q, out)


def test_norm_of_zero_row_is_zero():
    z = torch.zeros((1, 1, 128), dtype=BF, device="cuda")
    kc, vc, out = (torch.ones((1, 1, 16, 128), dtype=BF, device="cuda") for _ in range(3))
    w = torch.ones(128, dtype=BF, device="cuda")
    out = torch.ones((1, 1, 128), dtype=BF, device="cuda")
    qdk.think_norm_rope_append(z, z, z, w, w, 1e-6, None, False, i32([4]), torch.tensor([3], device="cuda"), out, kc, vc)
    assert not out.any() and not kc[0, 0, 3].any() and kc.sum().item() == 15 * 128


# ------------------------------------------------------------------ attention --

def run_attn(x: P.Batch, Hq, Hkv, max_new=0, out=None, workspace=None, scale=SCALE):
    w = attn_ws(x.T, Hq, Hkv, x.dtype) if workspace is None else workspace
    out = torch.full((x.T, Hq, 128), 9.0, dtype=x.dtype, device="cuda") if out is None else out
    qdk.think_paged_attn(x.q.cuda(), x.cache(x.k), x.cache(x.v), i32(x.table), i32(x.q_start), i32(x.lens), out, w,
                         window=x.window, scale=scale, max_new=max_new)
    assert qdk.think_read_device_status(w) == 0
    return out


def check_attn(x: P.Batch, Hq, Hkv, max_new=0, scale=SCALE):
    got = run_attn(x, Hq, Hkv, max_new, scale=scale).cpu().to(P.F64)
    want, size, logit = P.attend(x.q, x.k, x.v, x.table, x.q_start, x.lens, x.window, scale)
    inside = x.q_start[-1]
    assert (got[inside:] == 9.0).all(), "rows behind the last request were written"
    got, want, size, logit = got[:inside], want[:inside], size[:inside], logit[:inside]
    assert torch.isfinite(got).all()
    bound = P.attend_bound(want, size, logit, x.dtype, max(x.lens + [1]))
    over = (got - want).abs() / bound
    assert over.max().item() <= 1.0, f"error {over.max().item():.3g} of the bound at {over.argmax().item()}"


SHAPES = [
    # new, ctx, Hq, Hkv, page, window
    ([1], [0], 1, 1, 16, 0), ([1], [1], 4, 1, 16, 0), ([1], [700], 32, 8, 64, 0), ([1], [5000], 4, 1, 16, 0),
    ([1, 1, 1, 1, 1], [0, 127, 128, 129, 1000], 8, 2, 16, 0), ([3], [0], 4, 4, 32, 0), ([17], [3], 2, 1, 48, 0),
    ([128], [0], 4, 4, 64, 0), ([129], [0], 1, 1, 128, 0), ([300], [0], 4, 1, 16, 0), ([257], [300], 6, 2, 80, 0),
    ([64, 0, 1, 33, 0, 2], [10, 50, 400, 0, 0, 127], 8, 2, 32, 0), ([5, 70], [30, 0], 7, 1, 16, 0),
    ([40], [90], 12, 1, 256, 0), ([20, 1], [600, 900], 16, 2, 48, 0),
    ([1, 200, 1], [900, 100, 30], 8, 2, 16, 64), ([300], [0], 4, 2, 32, 100), ([2, 40], [400, 300], 4, 1, 64, 1),
    ([1, 1], [3000, 10], 8, 1, 16, 500), ([150], [500], 3, 1, 48, 333), ([600], [200], 2, 2, 112, 0),
    # many key tiles a block: one request's keys shared by all blocks, rows shared, several items a block, both kinds in turn
    ([1], [150000], 4, 1, 64, 0), ([3], [120000], 8, 1, 16, 90001), ([200], [40000], 2, 1, 128, 0),
    ([1] * 40, [37 * i for i in range(40)], 16, 8, 16, 0), ([1, 300, 2, 70, 1, 140] * 4, [900, 10, 3000, 200, 0, 1500] * 4, 8, 4, 32, 0),
    ([2, 260, 1, 33] * 6, [1400, 0, 700, 2100] * 6, 12, 4, 48, 600)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attn(i, dtype):
    new, ctx, Hq, Hkv, page, window = SHAPES[i]
    x = P.Batch(new, ctx, Hq, Hkv, page, dtype, 100 + i, window=window, layout="nhd" if i % 2 else "hnd", pad_rows=i % 3)
    check_attn(x, Hq, Hkv, max_new=max(new) if i % 4 else 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new,ctx", [
    ([1] * 12, [128 * n + d for n in (15, 16, 17) for d in (-2, -1, 0, 1)]),  # single tokens about 16 key tiles
    ([64, 33, 65, 130], [128 * 15, 128 * 16, 900, 1000]), ([70] * 6, [128 * 7, 128 * 7 + 58, 128 * 8, 1200, 60, 0]),
    ([1], [128 * 17]), ([1, 1, 400], [128 * 16 + 1, 5, 600])])
def test_attn_short_items_and_those_that_are_cut(new, ctx, dtype):
    check_attn(P.Batch(new, ctx, 8, 2, 32, dtype, 77 + len(new)), 8, 2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_rows_that_see_nothing(dtype):
    """Fewer tokens cached than new ones: the first rows have positions below 0 and get zeros."""
    x = P.Batch([6, 300, 4], [0, 0, 0], 4, 2, 16, dtype, 3, lens=[2, 170, 0])
    check_attn(x, 4, 2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_widest_window(dtype):
    """A window wider than any position hides nothing, rows before position 0 included."""
    x = P.Batch([6, 300], [0, 500], 4, 2, 16, dtype, 5, lens=[2, 800])
    want = run_attn(x, 4, 2)
    for x.window in (2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1):
        assert torch.equal(run_attn(x, 4, 2), want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_large_logits(dtype):
    """Sharp softmax: maxima that grow along the keys, and weights that underflow."""
    x = P.Batch([40, 1], [700, 900], 8, 2, 32, dtype, 4, key_scale=12.0)
    ramp = torch.linspace(0.02, 1.0, x.k.shape[0])[:, None, None, None]
    x.k = (x.k.float() * ramp).to(dtype)
    check_attn(x, 8, 2)
    check_attn(x, 8, 2, scale=-0.05)
    check_attn(x, 8, 2, scale=0.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv", [(6, 2), (8, 2)])
def test_attn_strides_and_views(dtype, Hq, Hkv):
    """q a view of a fused projection, out a view of a wider buffer, the table a view: canaries around stay."""
    x = P.Batch([33, 2], [100, 60], Hq, Hkv, 32, dtype, 8)
    wide = torch.full((x.T, Hq + 3, 192), 5.0, dtype=dtype, device="cuda")
    q = wide[:, 1:1 + Hq, 32:160]
    q.copy_(x.q)
    dst = torch.full((x.T + 2, Hq + 2, 256), 5.0, dtype=dtype, device="cuda")
    out = dst[1:1 + x.T, 1:1 + Hq, 64:192]
    tab = torch.full((3, len(x.table[0]) + 4), -1, dtype=torch.int32, device="cuda")
    tab[:2, 2:-2] = i32(x.table)
    w = attn_ws(x.T, Hq, Hkv, dtype)
    qdk.think_paged_attn(q, x.cache(x.k), x.cache(x.v), tab[:2, 2:-2], i32(x.q_start), i32(x.lens), out, w)
    assert torch.equal(out, run_attn(x, Hq, Hkv))
    out.fill_(5.0)
    assert (dst == 5.0).all()
    # one row of queries for all tokens and heads
    x.q[:] = x.q[:1, :1].clone()
    w = attn_ws(x.T, Hq, Hkv, dtype)
    qdk.think_paged_attn(x.q[:1, :1].cuda().expand(x.T, Hq, 128), x.cache(x.k), x.cache(x.v), i32(x.table), i32(x.q_start),
                         i32(x.lens), out, w)
    assert torch.equal(out, run_attn(x, Hq, Hkv))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad_page,pad_head", [(8, 0), (24, 40), (0, 8)])
def test_attn_pages_and_heads_at_any_distance(dtype, pad_page, pad_head):
    """Strides of pages and heads that are not multiples of one another."""
    x = P.Batch([3, 40], [600, 130], 6, 3, 32, dtype, 41)

    def spread(c):  # [pages,Hkv,page,128] with gaps of NaN behind each head and page
        n, h, rows, d = c.shape
        sh = rows * d + pad_head
        sp = h * sh + pad_page
        flat = torch.full((n * sp,), float("nan"), dtype=dtype, device="cuda")
        out = torch.as_strided(flat, c.shape, (sp, sh, d, 1))
        out.copy_(c)
        return out

    w = attn_ws(x.T, 6, 3, dtype)
    out = torch.full((x.T, 6, 128), 9.0, dtype=dtype, device="cuda")
    qdk.think_paged_attn(x.q.cuda(), spread(x.cache(x.k)), spread(x.cache(x.v)), i32(x.table), i32(x.q_start), i32(x.lens), out, w,
                         scale=SCALE)
    assert qdk.think_read_device_status(w) == 0
    assert torch.equal(out, run_attn(x, 6, 3))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hkv", [1, 2])
def test_attn_pool_of_one_page(dtype, Hkv):
    x = P.Batch([2], [10], 2 * Hkv, Hkv, 16, dtype, 43)
    page = x.table[0][0]
    w = attn_ws(x.T, 2 * Hkv, Hkv, dtype)
    out = torch.full((x.T, 2 * Hkv, 128), 9.0, dtype=dtype, device="cuda")
    qdk.think_paged_attn(x.q.cuda(), x.cache(x.k)[page:page + 1], x.cache(x.v)[page:page + 1],
                         i32([[0] + x.table[0][1:]]), i32(x.q_start), i32(x.lens), out, w, scale=SCALE)
    assert qdk.think_read_device_status(w) == 0
    assert torch.equal(out, run_attn(x, 2 * Hkv, Hkv))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_bad_pages_count_as_zeros(dtype):
    x = P.Batch([5, 40], [200, 90], 4, 2, 32, dtype, 9, poison=False)
    x.table[0][2], x.table[1][1] = -1, x.k.shape[0]
    w = attn_ws(x.T, 4, 2, dtype)
    out = torch.empty((x.T, 4, 128), dtype=dtype, device="cuda")
    qdk.think_paged_attn(x.q.cuda(), x.cache(x.k), x.cache(x.v), i32(x.table), i32(x.q_start), i32(x.lens), out, w)
    assert qdk.think_read_device_status(w) == qdk.THINK_DEVICE_BAD_PAGE
    pool = x.k.shape[0]
    zero = torch.zeros_like(x.k[:1])
    x.k, x.v = torch.cat([x.k, zero]), torch.cat([x.v, zero])
    x.table[0][2] = x.table[1][1] = pool
    assert torch.equal(out, run_attn(x, 4, 2))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_lengths_out_of_bounds_are_held(dtype):
    """Garbage in the device arrays stays inside the buffers."""
    x = P.Batch([8, 30], [100, 10], 4, 2, 16, dtype, 10, poison=False)
    w = attn_ws(x.T, 4, 2, dtype)
    canary = torch.full((x.T + 8, 4, 128), 5.0, dtype=dtype, device="cuda")
    out = canary[4:4 + x.T]
    for q_start, lens in (([0, 8, 10 ** 9], [10 ** 9, -4]), ([-50, 8, 3], [100, 2 ** 31 - 1]), ([40, 2, -1], [7, 40])):
        qdk.think_paged_attn(x.q.cuda(), x.cache(x.k), x.cache(x.v), i32(x.table), i32(q_start), i32(lens), out, w)
    torch.cuda.synchronize()
    assert (canary[:4] == 5.0).all() and (canary[4 + x.T:] == 5.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_repeats_bit_for_bit_and_shares_a_workspace(dtype):
    a = P.Batch([1, 90, 300], [2000, 10, 700], 8, 2, 32, dtype, 12)
    b = P.Batch([2], [4000], 4, 1, 16, dtype, 13)
    w = attn_ws(4096, 8, 1, dtype)
    outs = [(run_attn(a, 8, 2, workspace=w), run_attn(b, 4, 1, workspace=w)) for _ in range(3)]
    for p, q in outs[1:]:
        assert torch.equal(p, outs[0][0]) and torch.equal(q, outs[0][1])


def test_attn_many_requests():
    """More requests than a block has threads, some empty, and long tables."""
    r = random.Random(6)
    new = [r.choice([0, 1, 1, 2]) for _ in range(700)]
    ctx = [r.randint(0, 60) for _ in range(700)]
    x = P.Batch(new, ctx, 2, 1, 16, BF, 14)
    check_attn(x, 2, 1, max_new=2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_captured_follows_the_lengths(dtype):
    """One captured call, replayed after the lengths, rows and tables on the device changed."""
    Hq, Hkv = 8, 2
    xs = [P.Batch(n, c, Hq, Hkv, 16, dtype, 20 + i, pad_rows=80 - sum(n)) for i, (n, c) in enumerate(
        [([1, 1, 40], [300, 20, 7]), ([30, 1, 2], [0, 900, 640]), ([80, 0, 0], [0, 0, 5])])]
    pool, width = max(x.k.shape[0] for x in xs), max(len(x.table[0]) for x in xs)
    q = torch.zeros((80, Hq, 128), dtype=dtype, device="cuda")
    k = torch.zeros((pool, Hkv, 16, 128), dtype=dtype, device="cuda")
    v, out = torch.zeros_like(k), torch.zeros_like(q)
    tab, qs, lens = i32([[0] * width] * 3), i32([0] * 4), i32([1] * 3)
    w = attn_ws(80, Hq, Hkv, dtype)
    call = lambda: qdk.think_paged_attn(q, k, v, tab, qs, lens, out, w)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x in xs + xs[:1]:
        q.copy_(x.q)
        k[:x.k.shape[0]].copy_(x.k)
        v[:x.k.shape[0]].copy_(x.v)
        tab.fill_(-1)
        tab[:, :len(x.table[0])] = i32(x.table)
        qs.copy_(i32(x.q_start))
        lens.copy_(i32(x.lens))
        out.fill_(9.0)
        g.replay()
        assert torch.equal(out, run_attn(x, Hq, Hkv))


# ------------------------------------------------------------------ page gather --

@pytest.mark.parametrize("dtype,page,layout,lens,N", [
    (BF, 16, "hnd", [1], 1), (BF, 64, "nhd", [1000, 0, 333], 1000), (F32, 48, "hnd", [97, 500], 301), (F32, 256, "nhd", [700], 900)])
def test_gather_pages(dtype, page, layout, lens, N):
    x = P.Batch([0] * len(lens), lens, 3, 3, page, dtype, N, layout=layout)
    want = torch.zeros((len(lens), 3, N, 128), dtype=dtype)
    for b, n in enumerate(lens):
        for j in range(min(n, N)):
            want[b, :, j] = x.k[x.table[b][j // page], :, j % page]
    canary = torch.full((want.numel() + 256,), 5.0, dtype=dtype, device="cuda")
    out = canary[128:-128].view(want.shape)
    qdk.think_gather_pages(x.cache(x.k), i32(x.table), i32(x.lens), out)
    assert torch.equal(out.cpu(), want)
    assert (canary[:128] == 5.0).all() and (canary[-128:] == 5.0).all()


def test_gather_bad_pages_and_lengths_give_zeros():
    x = P.Batch([0, 0], [40, 40], 2, 2, 16, BF, 1, poison=False)
    x.table[0][1], x.table[1][0] = -3, x.k.shape[0]
    out = torch.full((2, 2, 100, 128), 9.0, dtype=BF, device="cuda")
    qdk.think_gather_pages(x.cache(x.k), i32(x.table), i32([-5, 2 ** 31 - 1]), out)
    assert not out[0].any()
    assert not out[1, :, :16].any() and torch.equal(out[1, :, 16:40].cpu(), torch.cat(
        [x.k[x.table[1][1]], x.k[x.table[1][2]][:, :8]], 1))
    assert not out[1, :, len(x.table[0]) * 16:].any()


# ------------------------------------------------------------------ streams --

def test_two_streams_at_once():
    xs = [P.Batch([50, 1], [400, 1500], 8, 2, 16, BF, 30 + i) for i in range(2)]
    want = [run_attn(x, 8, 2) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    args = [(x.q.cuda(), x.cache(x.k), x.cache(x.v), i32(x.table), i32(x.q_start), i32(x.lens), torch.zeros_like(o),
             attn_ws(x.T, 8, 2, BF)) for x, o in zip(xs, want)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, a in zip(streams, args):
            qdk.think_paged_attn(*a, stream=s)
    torch.cuda.synchronize()
    for a, o in zip(args, want):
        assert torch.equal(a[6], o)


# ------------------------------------------------------------- the calls together --

def serve(cache, steps, Hq, Hkv, dtype, seed, freq, window):
    """Run steps of new tokens through a PagedCache and check every call against plain fp64 on what the pages hold."""
    g = torch.Generator().manual_seed(seed)
    wq, wk = (1 + 0.2 * torch.randn((2, 128), generator=g)).to(dtype)
    B = cache.B
    lens, rows_seen = [0] * B, [[] for _ in range(B)]
    for new in steps:
        T = sum(new) + 3
        qkv = torch.randn((T, Hq + 2 * Hkv, 128), generator=g).to(dtype)
        dev = qkv.cuda()
        q_out, out = (torch.full((T, Hq, 128), 9.0, dtype=dtype, device="cuda") for _ in range(2))
        cache.extend(i32(new), rows=T)
        cache.append(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], q_out, wq.cuda(), wk.cuda(), 1e-6, freq, layer=1)
        cache.attend(q_out, out, window=window, max_new=max(new), layer=1)
        lens = [a + n for a, n in zip(lens, new)]
        assert cache.kv_lens.tolist() == lens
        q_start = [0]
        for n in new:
            q_start.append(q_start[-1] + n)
        # keys and values where the tables say, at their positions
        table, k_cache, v_cache = cache.block_table.tolist(), cache.k_cache[1].cpu(), cache.v_cache[1].cpu()
        for b, n in enumerate(new):
            pos = torch.arange(lens[b] - n, lens[b])
            yk, sk = P.turned(qkv[q_start[b]:q_start[b + 1], Hq:Hq + Hkv], wk, 1e-6, freq.cpu(), False, pos)
            for i, p in enumerate(pos.tolist()):
                page, row = table[b][p // cache.page_size], p % cache.page_size
                assert torch.equal(v_cache[page, :, row], qkv[q_start[b] + i, Hq + Hkv:])
                err = (k_cache[page, :, row].to(P.F64) - yk[i]).abs()
                assert (err <= 90 * 2.0 ** -24 * sk[i] + P.HALF_STEP[dtype] * (1 + 2.0 ** -6) * yk[i].abs() + 1e-30).all()
        want, size, logit = P.attend(q_out[:T - 3].cpu(), k_cache, v_cache, table, q_start, lens, window, SCALE)
        got = out.cpu().to(P.F64)
        assert (got[T - 3:] == 9.0).all()
        assert ((got[:T - 3] - want).abs() <= P.attend_bound(want, size, logit, dtype, max(lens + [1]))).all()
        for b in range(B):
            rows_seen[b].append(q_out[q_start[b]:q_start[b + 1]].cpu())
    assert qdk.think_read_device_status(cache.extend_ws) == 0 and qdk.think_read_device_status(cache.attn_ws) == 0
    return lens, rows_seen


@pytest.mark.parametrize("dtype,window", [(BF, 0), (F32, 0), (BF, 100)])
def test_prompts_then_decode_then_prune(dtype, window):
    """Prompt chunks and single tokens of three requests through the pages; one is released and its pages serve a new
    request; one is handed to the channel pruning and decoded from the thinner cache."""
    import numpy as np
    import oracle
    Hq, Hkv, page = 8, 2, 32
    cache = qdk.PagedCache(3, Hq, Hkv, num_pages=40, page_size=page, max_blocks=16, max_rows=512, layers=2, dtype=dtype)
    freq = (10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).cuda()
    lens, rows = serve(cache, [[200, 0, 31], [97, 1, 1], [1, 130, 1], [1, 1, 1]], Hq, Hkv, dtype, 3, freq, window)
    assert lens == [299, 132, 34] and cache.free_count.item() == 40 - 10 - 5 - 2
    N, T = lens[0], 77
    q_win = rows[0][1][-32:].transpose(0, 1)[None].contiguous()  # the last 32 queries of its second chunk
    pruned, v = cache.prune(0, N, q_win.cuda(), T, layer=1)
    k, _ = cache.gather(0, N, layer=1)
    f64 = lambda t: t.cpu().to(torch.float64).numpy()
    scores, idx, kp = oracle.oracle_prune(f64(q_win), f64(k), T)
    from helpers import check_out, idx_mismatch_heads, kp_logical
    assert not idx_mismatch_heads(pruned.idx.cpu().numpy(), idx, scores, T)
    assert np.array_equal(kp_logical(pruned.k_pruned, N), kp)
    q = torch.randn((1, Hq, 128), generator=torch.Generator().manual_seed(1)).to(dtype)
    out = torch.empty((1, Hq, 128), dtype=torch.float32, device="cuda")
    pruned.decode(q.cuda(), v, out)
    check_out(out, oracle.oracle_decode(f64(q), kp, f64(v), idx), dtype)
    cache.release(0)
    assert cache.free_count.item() == 33 and cache.kv_lens.tolist() == [0, 132, 34]
    held = [p for b in (1, 2) for p in cache.block_table[b].tolist() if p >= 0]
    assert sorted(held + cache.free_pages[:33].tolist()) == list(range(40))


def test_step_captured_and_replayed():
    """Tables, write and attention of a decode step in one graph: replays advance the requests."""
    Hq, Hkv, page, B = 8, 2, 16, 4
    def fresh():
        cache = qdk.PagedCache(B, Hq, Hkv, num_pages=64, page_size=page, max_blocks=16, max_rows=B)
        return cache, torch.zeros((B, Hq, 128), dtype=BF, device="cuda"), torch.zeros((B, Hq, 128), dtype=BF, device="cuda")
    freq = (10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).cuda()
    one = i32([1] * B)
    qkv = torch.zeros((B, Hq + 2 * Hkv, 128), dtype=BF, device="cuda")

    def step(c, q_out, out):
        c.extend(one)
        c.append(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], q_out, inv_freq=freq)
        c.attend(q_out, out, max_new=1)

    inputs = [torch.randn(qkv.shape, generator=torch.Generator().manual_seed(i)).to(BF).cuda() for i in range(40)]
    a, b = fresh(), fresh()
    want = []
    for x in inputs:
        qkv.copy_(x)
        step(*a)
        want.append(a[2].clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*b)
    for x, w in zip(inputs, want):
        qkv.copy_(x)
        graph.replay()
        assert torch.equal(b[2], w)
    assert b[0].kv_lens.tolist() == [40] * B and torch.equal(a[0].block_table, b[0].block_table)


@pytest.mark.parametrize("what", ["extend", "rope", "attn", "gather"])
def test_binding_refusals_on_the_gpu(what):
    """Shapes and types that do not match are refused before any launch."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    l = lambda *s: torch.zeros(s, dtype=torch.int64, device="cuda")
    h = lambda *s: torch.zeros(s, dtype=BF, device="cuda")
    w = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    if what == "extend":
        good = [i(3), i(3), i(3, 4), i(9), i(1), 16, i(3), i(1), i(4), i(5), l(5), w]
        bad = {0: i(4), 1: l(3), 2: i(4, 4), 3: i(3, 3), 4: i(2), 5: "x", 6: i(2), 7: i(0), 8: i(3), 9: l(5), 10: i(5),
               11: w[::2]}
        call = qdk.think_extend_pages
    elif what == "rope":
        good = [h(5, 4, 128), h(5, 2, 128), h(5, 2, 128), h(128), h(128), 1e-6, torch.zeros(64, dtype=torch.float64, device="cuda"),
                False, i(5), l(5), h(5, 4, 128), h(3, 2, 16, 128), h(3, 2, 16, 128)]
        bad = {0: h(5, 4, 128).float(), 1: h(4, 2, 128), 2: h(5, 3, 128), 3: h(64), 4: h(128).float(), 5: "x",
               6: torch.zeros(64, device="cuda"), 7: torch.zeros(2), 8: l(5), 9: i(5), 10: h(5, 4, 64), 11: h(3, 1, 16, 128), 12: h(3, 2, 16, 128)[:2]}
        call = qdk.think_norm_rope_append
    elif what == "attn":
        good = [h(5, 4, 128), h(3, 2, 16, 128), h(3, 2, 16, 128), i(2, 4), i(3), i(2), h(5, 4, 128),
                torch.zeros(qdk.think_paged_attn_workspace_size(5, 4, 2), dtype=torch.uint8, device="cuda")]
        bad = {0: h(5, 4, 128).float(), 1: h(3, 2, 16, 64), 2: h(2, 2, 16, 128), 3: l(2, 4), 4: i(2), 5: i(4)[::2],
               6: h(4, 4, 128), 7: torch.zeros(256, dtype=torch.uint8, device="cuda")}
        call = qdk.think_paged_attn
    else:
        good = [h(3, 2, 16, 128), i(2, 4), i(2), h(2, 2, 9, 128)]
        bad = {0: h(3, 2, 16, 128).float(), 1: i(3, 4), 2: l(2), 3: h(2, 2, 9, 256)[..., ::2]}
        call = qdk.think_gather_pages
    call(*good)
    for at, x in bad.items():
        args = list(good)
        args[at] = x
        with pytest.raises(qdk.ThinkError):
            call(*args)
