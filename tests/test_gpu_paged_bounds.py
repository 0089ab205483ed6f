"""The attention over pages on the GPU, held to the bounds of paged_bounds."""
import math

import pytest
import torch

import paged_bounds as Q

pytestmark = pytest.mark.gpu
qdk = pytest.importorskip("query_driven_key_b200")

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
SCALE = 1.0 / math.sqrt(128.0)


def attend(q, k, v, table, q_start, lens, window=0, scale=SCALE):
    """think_paged_attn on CPU or GPU tensors, lists for the integers; the status word has to be 0."""
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    T, Hq, _ = q.shape
    w = torch.full((qdk.think_paged_attn_workspace_size(T, Hq, k.shape[1], dtype=q.dtype),), 255, dtype=torch.uint8, device="cuda")
    w[:256 + 2048] = 0  # (only the status word and the counters have to be zero: the scratch holds NaN)
    out = torch.full_like(q, 9.0)
    qdk.think_paged_attn(q, k, v, i32(table), i32(q_start), i32(lens), out, w, window=window, scale=scale)
    assert qdk.think_read_device_status(w) == 0
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(Q.LONG)))
def test_long_contexts(i, dtype):
    Hq, Hkv, window = Q.LONG[i][2], Q.LONG[i][3], Q.LONG[i][5]
    x = Q.long_batch(i, dtype)
    want, size, spread, logit = Q.exact(x, SCALE)
    limit = Q.bound(want, size, spread, logit, dtype, Q.chain(x, Hq, Hkv))
    got = attend(x.q, x.cache(x.k), x.cache(x.v), x.table, x.q_start, x.lens, window).cpu().to(F64)
    assert ((got - want).abs() / limit).max().item() <= 1.0


@pytest.mark.parametrize("keys", [3000, 20000])
def test_fp32_mean_of_positive_values(keys):
    """Nearly equal weights over one long item a block: what the sums of O drop would all have one sign."""
    B, page = Q.PARTS, 64
    cols = -(-keys // page)
    g = torch.Generator(device="cuda").manual_seed(1)
    v = torch.rand((B * cols, 1, page, 128), generator=g, device="cuda") + 0.5
    k = torch.randn((B * cols, 1, page, 128), generator=g, device="cuda")
    table = torch.randperm(B * cols, generator=g, device="cuda").reshape(B, cols)
    q = 0.01 * torch.randn((B, 1, 128), generator=g, device="cuda")
    got = attend(q, k, v, table, list(range(B + 1)), [keys] * B).to(F64)
    for b in range(B):
        kk, vv = (c[table[b], 0].reshape(-1, 128)[:keys].to(F64) for c in (k, v))
        want = torch.softmax(SCALE * (q[b].to(F64) @ kk.T), -1) @ vv
        limit = Q.mean_bound(-(-keys // 64), SCALE * (q[b].to(F64).abs() @ kk.abs().T).max().item())
        assert ((got[b] - want).abs() / want).max().item() <= limit, b


@pytest.mark.parametrize("B,G", [(148, 1), (100, 2), (148, 160)])
def test_bf16_sums_over_long_items_do_not_drift(B, G):
    """200000 keys a request and positive values: keys shared by the halves of a block, in one piece and cut, and rows
    shared.  Of 8 * 256 steps between two roundings to nearest each drops at most 2 u; the mean over all outputs leaves
    6 standard deviations of a rounding, 2^-8 / sqrt(3), of this result and of the exact one."""
    keys, page, pool = 200000, 64, 64
    g = torch.Generator(device="cuda").manual_seed(B + G)
    v = (torch.rand((pool, 1, page, 128), generator=g, device="cuda") + 0.5).to(BF)
    k = torch.randn((pool, 1, page, 128), generator=g, device="cuda").to(BF)
    q = torch.randn((B, G, 128), generator=g, device="cuda").to(BF)
    table = torch.randint(0, pool, (B, keys // page), generator=g, device="cuda")
    got = attend(q, k, v, table, list(range(B + 1)), [keys] * B).to(F64)
    want = torch.empty_like(got)
    for b in range(B):
        e = torch.exp(SCALE * (q[b].to(F64) @ k.reshape(-1, 128).to(F64).T))
        e = e * torch.bincount(table[b], minlength=pool).repeat_interleave(page)
        want[b] = e @ v.reshape(-1, 128).to(F64) / e.sum(-1, keepdim=True)
    drift = ((got - want.to(BF).to(F64)) / want).mean().item()
    assert abs(drift) <= 8 * 256 * 2 * Q.U + 6 * 2.0 ** -8 / math.sqrt(3.0) * math.sqrt(2.0 / got.numel())
    assert ((got - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want).all()


def test_fp32_values_keep_their_third_part():
    v = Q.with_third_part((1 + torch.rand((3, 1, 512, 128), generator=torch.Generator().manual_seed(2)) / 2).to(BF))
    v[:] = v[:, :, :1]  # every row the same: the mean is the row
    k = torch.randn(v.shape, generator=torch.Generator().manual_seed(4))
    got = attend(torch.zeros(1, 1, 128), k, v[:1].expand(3, -1, -1, -1).contiguous(), [[2, 0, 1]], [0, 1], [1200]).cpu().to(F64)
    want = v[0, 0, 0].to(F64)
    assert ((got[0, 0] - want).abs() / want).max().item() <= Q.mean_bound(20)


def test_fp32_logits_keep_their_third_parts():
    q, k0 = Q.two_key_case()
    B = len(q)
    qq, k, v = torch.zeros(B, 1, 128), torch.zeros(B, 1, 16, 128), torch.zeros(B, 1, 16, 128)
    qq[:, 0, 5], k[:, 0, 0, 5] = q, k0
    v[:, 0, 0], v[:, 0, 1] = 1.0, -1.0
    got = attend(qq, k, v, [[b] for b in range(B)], list(range(B + 1)), [2] * B, scale=1.0).cpu().to(F64)
    want, limit = Q.two_key_want(q, k0), Q.two_key_bound(q, k0)
    assert ((got[:, 0] - want[:, None]).abs() / limit[:, None]).max().item() <= 1.0


def test_fp32_numbers_beyond_the_largest_bf16_one():
    """Finite numbers that round to infinity in bf16, as values and as keys; infinite values spoil their channel alone."""
    top = torch.finfo(F32).max
    v = torch.zeros(1, 1, 16, 128)
    v[0, 0, 0] = top * (1 - torch.arange(128) * 2.0 ** -14)
    v[0, 0, 0, 64:] *= -1
    got = attend(torch.randn(1, 1, 128), torch.randn(1, 1, 16, 128), v, [[0]], [0, 1], [1]).cpu().to(F64)
    want = v[0, 0, 0].to(F64)
    assert ((got[0, 0] - want) / want).abs().max().item() <= Q.mean_bound(1)
    v[0, 0, 0, 7], v[0, 0, 0, 70] = math.inf, -math.inf
    got = attend(torch.randn(1, 1, 128), torch.randn(1, 1, 16, 128), v, [[0]], [0, 1], [1]).cpu()
    fine = torch.ones(128, dtype=torch.bool)
    fine[[7, 70]] = False
    assert (got[0, 0].isfinite() == fine).all()
    q, k, v = torch.zeros(2, 1, 128), torch.zeros(2, 1, 16, 128), torch.zeros(2, 1, 16, 128)
    q[:, 0, 5], k[:, 0, 0, 5] = torch.tensor([2.0 ** -126, -(2.0 ** -126)]), torch.tensor([top, -top])
    v[:, 0, 0], v[:, 0, 1] = 1.0, -1.0
    got = attend(q, k, v, [[0], [1]], [0, 1, 2], [2, 2], scale=1.0).cpu().to(F64)
    a, b = q[:, 0, 5].abs(), k[:, 0, 0, 5].abs()
    assert ((got[:, 0] - Q.two_key_want(a, b)[:, None]).abs() <= Q.two_key_bound(a, b)[:, None]).all()
