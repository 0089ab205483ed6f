"""CPU: outputs that are wrong are outside the bounds of paged_bounds, and right ones inside."""
import math

import pytest
import torch

import paged_bounds as Q
import paged_plain as P

F32, BF, F64 = torch.float32, torch.bfloat16, torch.float64
SCALE = 1.0 / math.sqrt(128.0)


def worst(got, want, limit):
    return ((got - want).abs() / limit).max().item()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(Q.LONG)))
def test_long_contexts(i, dtype):
    new, ctx, Hq, Hkv, page, window = Q.LONG[i]
    x = Q.long_batch(i, dtype)
    want, size, spread, logit = Q.exact(x, SCALE)
    limit = Q.bound(want, size, spread, logit, dtype, Q.chain(x, Hq, Hkv))
    assert worst(want.to(dtype).to(F64), want, limit) <= 1.0
    assert worst(torch.zeros_like(want), want, limit) > 3.0
    # what one of 148 blocks does is lost: its keys count as if they were not there
    b = max(range(len(ctx)), key=lambda r: ctx[r])
    seen = min(x.lens[b], x.window) if window else x.lens[b]
    share = seen // Q.PARTS // page * page
    first = (x.lens[b] - seen // 2) // page
    lost = [p for p in x.table[b][first:first + share // page]]
    x.v = x.v.clone()
    x.v[lost] = 0
    without, _, _ = P.attend(x.q, x.k, x.v, x.table, x.q_start, x.lens, window, SCALE)
    assert worst(without, want, limit) > 1.5


def test_two_key_outputs_need_three_parts():
    q, k = Q.two_key_case()
    want, limit = Q.two_key_want(q, k), Q.two_key_bound(q, k)
    form = lambda a, b: torch.tanh(a * b / 2).to(F32).to(F64)
    assert worst(form(Q.parts_of(q, 3), Q.parts_of(k, 3)), want, limit) <= 1.0
    assert worst(form(Q.parts_of(q, 2), Q.parts_of(k, 3)), want, limit) > 1.0
    assert worst(form(Q.parts_of(q, 3), Q.parts_of(k, 2)), want, limit) > 1.0


def test_means_need_three_parts_and_short_sums():
    v = Q.with_third_part(torch.tensor([1.25], dtype=BF))
    assert abs(Q.parts_of(v, 2).item() / v.item() - 1) > Q.mean_bound(20)
    # one sum over 20000 keys, 16 a step, that drops what is below its last place
    total, step = 0.0, 16 * 1.2345678
    for _ in range(20000 // 16):
        s = total + step
        e = math.floor(math.log2(s)) - 23
        total = math.floor(s / 2.0 ** e) * 2.0 ** e
    assert 1 - total / 20000 / 1.2345678 > Q.mean_bound(313, 0.2)
