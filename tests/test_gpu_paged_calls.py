"""Calls of the paged cache that meet other threads, streams, refusals and extreme values, on the GPU."""
import math
import threading

import pytest
import torch

import paged_plain as P

pytestmark = pytest.mark.gpu
qdk = pytest.importorskip("query_driven_key_b200")

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def test_a_small_call_of_another_thread_does_not_take_shared_memory_away():
    """A prompt's rotation takes twice the shared memory of a single token's by the same kernel."""
    def call(T):
        x = torch.zeros((T, 32, 128), dtype=BF, device="cuda")
        cache = torch.zeros((2, T // 16 + 1, 8, 16, 128), dtype=BF, device="cuda")
        qdk.think_norm_rope_append(x[:, :16], x[:, 16:24], x[:, 24:], None, None, 0.0, None, False,
                                   torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda"),
                                   torch.empty_like(x[:, :16]), cache[0], cache[1])
    call(8192)
    failed = []

    def other():
        try:
            call(1)
        except Exception as e:
            failed.append(e)
    t = threading.Thread(target=other)
    t.start()
    t.join()
    assert not failed
    call(8192)
    torch.cuda.synchronize()


def filled(lens, Hq=8, Hkv=2, dtype=BF, page=32, seed=0, **kw):
    """A PagedCache with these lengths, the queries of its tokens and the inputs' keys and values."""
    need = sum(-(-n // page) for n in lens)
    cache = qdk.PagedCache(len(lens), Hq, Hkv, num_pages=need + 8, page_size=page, max_blocks=max(lens) // page + 4,
                           max_rows=sum(lens), dtype=dtype, **kw)
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((sum(lens), Hq + 2 * Hkv, 128), generator=g).to(dtype).cuda()
    q_out = torch.empty((sum(lens), Hq, 128), dtype=dtype, device="cuda")
    cache.extend(torch.tensor(lens, dtype=torch.int32, device="cuda"))
    cache.append(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], q_out)
    return cache, q_out, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]


class RawStream:
    """Another library's stream object: only its handle."""

    def __init__(self, s):
        self.cuda_stream = s.cuda_stream


@pytest.mark.parametrize("raw", [False, True])
def test_prune_and_gather_on_a_side_stream(raw):
    """With the current stream busy: what prune allocates and clears has to be in the side stream's order, and memory
    that it drops must not come back to the current stream's work before the side stream is done with it."""
    cache, q, _, _ = filled([700, 300])
    q_win = q[668:700].transpose(0, 1)[None].contiguous()
    want, want_v = cache.prune(0, 700, q_win, 64)
    want_k, _ = cache.gather(1, 300)
    torch.cuda.synchronize()
    current, side = torch.cuda.current_stream(), torch.cuda.Stream()
    for _ in range(3):
        dirt = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(40)]
        del dirt
        torch.cuda._sleep(20_000_000)  # about 10 ms
        s = RawStream(side) if raw else side
        got, v = cache.prune(0, 700, q_win, 64, stream=s)
        k, _ = cache.gather(1, 300, stream=s)
        later = [torch.full_like(k, 7.0) for _ in range(8)] + [torch.full_like(v, 7.0) for _ in range(8)]
        side.synchronize()
        assert torch.cuda.current_stream() == current
        assert qdk.think_read_device_status(got.score_ws, side) == 0
        with torch.cuda.stream(side):
            assert torch.equal(got.idx, want.idx) and torch.equal(got.k_pruned[..., :700], want.k_pruned[..., :700])
            assert torch.equal(v, want_v) and torch.equal(k, want_k)
        del later
    torch.cuda.synchronize()
    side.wait_stream(current)
    cache.release(0, stream=RawStream(side) if raw else side)
    side.synchronize()
    assert cache.kv_lens.tolist() == [0, 300] and cache.free_count.item() == 22 + 8


@pytest.mark.parametrize("dtype", [BF, F32])
def test_generate_after_the_hand_over(dtype):
    """A pruned prompt grows by more tokens than its rows are padded by, each decoded against the oracle."""
    import oracle
    from helpers import check_out
    N, more, T, Hq, Hkv = 301, 13, 51, 8, 2
    cache, q, k, v = filled([40, N + more], dtype=dtype, seed=7)
    cache.kv_lens[1] = N  # the rest comes token by token
    q_win = q[40 + N - 32:40 + N].transpose(0, 1)[None].contiguous()
    pruned, values = cache.prune(1, N, q_win, T, capacity=N + more)
    assert values.shape == (1, Hkv, N + more, 128) and not values[:, :, N:].any()
    keys, _ = cache.gather(1, N)
    f64 = lambda t: t.cpu().to(F64).numpy()
    for i in range(more):
        row = 40 + N + i
        new = k[row].reshape(1, Hkv, 1, 128).contiguous()
        keys = torch.cat([keys, new], 2)
        values[:, :, pruned.n] = v[row]
        pruned.append(new)
        assert pruned.n == N + i + 1
        out = torch.empty((1, Hq, 128), dtype=F32, device="cuda")
        pruned.decode(q[row:row + 1], values, out)
        idx = pruned.idx.cpu().numpy()
        kp = f64(keys.gather(3, pruned.idx.long()[:, :, None].expand(-1, -1, pruned.n, -1)))
        check_out(out, oracle.oracle_decode(f64(q[row:row + 1]), kp, f64(values[:, :, :pruned.n]), idx), dtype)
    assert qdk.think_read_device_status(pruned.decode_ws) == 0
    with pytest.raises(qdk.ThinkError):
        pruned.append(torch.zeros((1, Hkv, 64, 128), dtype=dtype, device="cuda"))


def test_a_refused_request_beside_others_and_again():
    """Three requests of which the second finds no pages: the others' rows are right, its own have slot -1 and the status
    tells; nothing of it is in the cache, and its tokens go in when another request has left."""
    Hq, Hkv, page = 4, 2, 16
    cache = qdk.PagedCache(3, Hq, Hkv, num_pages=7, page_size=page, max_blocks=8, max_rows=128)
    g = torch.Generator().manual_seed(2)

    def step(new):
        T = sum(new)
        qkv = torch.randn((T, Hq + 2 * Hkv, 128), generator=g).to(BF)
        dev = qkv.cuda()
        q_out, out = (torch.full((T, Hq, 128), 9.0, dtype=BF, device="cuda") for _ in range(2))
        cache.extend(torch.tensor(new, dtype=torch.int32, device="cuda"), rows=T)
        cache.append(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], q_out)
        cache.attend(q_out, out)
        return qkv, out.cpu()

    def check(qkv, out, requests):
        starts = cache.q_start.tolist()
        want, size, logit = P.attend(qkv[:, :Hq], cache.k_cache[0].cpu(), cache.v_cache[0].cpu(), cache.block_table.tolist(),
                                     starts, [n if b in requests else 0 for b, n in enumerate(cache.kv_lens.tolist())], 0,
                                     1 / math.sqrt(128))
        limit = P.attend_bound(want, size, logit, BF, 128)
        for b in requests:
            rows = slice(starts[b], starts[b + 1])
            assert ((out[rows].to(F64) - want[rows]).abs() <= limit[rows]).all()

    check(*step([40, 20, 10]), (0, 1, 2))  # 3, 2 and 1 pages
    assert cache.status() == 0
    before = [c.clone() for c in (cache.k_cache[0], cache.v_cache[0], cache.block_table, cache.free_count)]
    qkv, out = step([4, 30, 1])            # the second wants 2 pages of 1
    assert cache.kv_lens.tolist() == [44, 20, 11] and cache.q_start.tolist() == [0, 4, 34, 35]
    assert (cache.slots[4:34] == -1).all() and (cache.slots[:4] >= 0).all() and (cache.slots[34:] >= 0).all()
    check(qkv, out, (0, 2))
    assert torch.equal(before[2], cache.block_table) and torch.equal(before[3], cache.free_count)
    written = (cache.k_cache[0] != before[0]).any(-1).sum().item()
    assert written == 5 * Hkv
    assert cache.status() == qdk.THINK_DEVICE_NO_PAGES and cache.status() == 0
    cache.release(2)
    check(*step([0, 30, 0]), (1,))
    assert cache.kv_lens.tolist() == [44, 50, 0] and cache.status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("rot", [0, 32, 96, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(3, 2, 1), (40, 40, 4), (2600, 1, 1)])
def test_infinities_stay_in_their_channels(T, Hq, Hkv, rot, neighbours, dtype):
    """Without a norm, channels that are not turned are copied bit for bit, infinities and NaN among them, and a turned pair
    is spoilt by its own two channels alone."""
    g = torch.Generator().manual_seed(rot + T)
    qkv = torch.randn((T, Hq + 2 * Hkv, 128), generator=g).to(dtype)
    hit = torch.rand(qkv.shape, generator=g) < 0.05
    odd = torch.tensor([math.inf, -math.inf, math.nan, -0.0])[torch.randint(0, 4, qkv.shape, generator=g)]
    qkv = torch.where(hit, odd, qkv).to(dtype)
    dev = qkv.cuda()
    freq = None if rot == 0 else (100.0 ** (-torch.arange(0, rot, 2, dtype=F64) / rot)).cuda()
    pos = torch.randint(1, 1000, (T,), generator=g).to(torch.int32)
    pages = -(-T // 16)
    kc, vc = (torch.zeros((pages, Hkv, 16, 128), dtype=dtype, device="cuda") for _ in range(2))
    q_out = torch.zeros((T, Hq, 128), dtype=dtype, device="cuda")
    qdk.think_norm_rope_append(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], None, None, 0.0, freq, neighbours,
                               pos.cuda(), torch.arange(T, device="cuda"), q_out, kc, vc)
    rows = lambda c: c.cpu().transpose(1, 2).reshape(-1, Hkv, 128)[:T]
    bits = lambda t: t.contiguous().view(torch.int16 if dtype == BF else torch.int32)
    got = torch.cat([q_out.cpu(), rows(kc)], 1)
    x = qkv[:, :Hq + Hkv]
    same = (bits(got[..., rot:]) == bits(x[..., rot:])) | (got[..., rot:].isnan() & x[..., rot:].isnan())
    assert same.all()
    assert torch.equal(bits(rows(vc)), bits(qkv[:, Hq + Hkv:]))
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + rot // 2)
        fine = x[..., a].isfinite() & x[..., b].isfinite()
        assert (got[..., a].isfinite() == fine).all() and (got[..., b].isfinite() == fine).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_pool_of_more_than_2_to_the_32_elements(dtype):
    """The last pages of pools whose offsets pass 32 bits: written, attended over and gathered like those of a small pool."""
    Hq, Hkv, page, pages, n = 4, 2, 64, 300_000, 150
    g = torch.Generator().manual_seed(8)
    x = torch.randn((n, Hq + 2 * Hkv, 128), generator=g).to(dtype).cuda()
    freq = (10000.0 ** (-torch.arange(0, 128, 2, dtype=F64) / 128)).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    lens, rows = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    results = []
    for total in (3, pages):
        kc, vc = (torch.empty((total, Hkv, page, 128), dtype=dtype, device="cuda") for _ in range(2))
        table = torch.tensor([[total - 1, total - 3, total - 2]], dtype=torch.int32, device="cuda")
        slots = table[0, pos.long() // page].long() * page + pos.long() % page
        q_out, out = torch.empty_like(x[:, :Hq]), torch.empty((n, Hq, 128), dtype=dtype, device="cuda")
        qdk.think_norm_rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], None, None, 0.0, freq, False, pos, slots, q_out, kc, vc)
        w = torch.zeros(qdk.think_paged_attn_workspace_size(n, Hq, Hkv, dtype=dtype), dtype=torch.uint8, device="cuda")
        qdk.think_paged_attn(q_out, kc, vc, table, rows, lens, out, w)
        assert qdk.think_read_device_status(w) == 0
        keys = torch.empty((1, Hkv, n, 128), dtype=dtype, device="cuda")
        qdk.think_gather_pages(kc, table, lens, keys)
        results.append((out, keys, vc[-1].clone()))
        del kc, vc
    assert pages * Hkv * page * 128 > 2 ** 32 and results[0][0].isfinite().all()
    for a, b in zip(*results):
        assert torch.equal(a, b)
    torch.cuda.empty_cache()
