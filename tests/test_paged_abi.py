"""CPU checks of the paged cache's entry points: sizes, and every refusal.  No kernel is launched: each call is rejected by
host validation, has nothing to do, or is a pure host function."""
import ctypes

import pytest
import torch

qdk = pytest.importorskip("query_driven_key_b200")
lib = qdk.lib

FAKE = ctypes.c_void_p(0x10000)        # never dereferenced: validation rejects first
ODD = ctypes.c_void_p(0x10002)
OFF8 = ctypes.c_void_p(0x10008)
OK, ARG, UNSUP, WS, ALIGN = (qdk.THINK_OK, qdk.THINK_ERR_INVALID_ARG, qdk.THINK_ERR_UNSUPPORTED, qdk.THINK_ERR_WORKSPACE,
                             qdk.THINK_ERR_ALIGNMENT)


def i64(*x):
    return (ctypes.c_int64 * len(x))(*x)


def caller(fn, **defaults):
    names = list(defaults)

    def call(**kw):
        assert set(kw) <= set(names), kw
        return fn(*dict(defaults, **kw).values(), None)
    return call


def test_sizes():
    assert qdk.think_extend_pages_workspace_size() == 256
    size = qdk.think_paged_attn_workspace_size
    assert size(1, 32, 8) < size(16, 32, 8) < size(32, 32, 8) == size(4096, 32, 8) == size(4096, 8, 8)
    assert 0 < size(64, 8, 8, dtype=torch.float32) < size(128, 8, 8, dtype=torch.float32) == size(5000, 32, 8, dtype=torch.float32) < size(4096, 8, 8)
    assert size(10, 30, 8) == 0 and size(10, 32, 8, d=64) == 0 and size(10, 4, 8) == 0


def test_extend_refusals():
    f = caller(lib.think_extend_pages, new=FAKE, lens=FAKE, B=2, page=16, table=FAKE, ld=8, blocks=8, free=FAKE, n_free=9,
               count=FAKE, T=10, lens_out=FAKE, count_out=FAKE, q_start=FAKE, pos=FAKE, slots=FAKE, ws=FAKE, bytes=256)
    assert f(B=-1) == ARG and f(T=-1) == ARG and f(n_free=-1) == ARG and f(page=0) == ARG and f(blocks=0) == ARG
    assert f(ld=7) == ARG and f(table=None) == ARG
    for name in ("new", "lens", "count", "lens_out", "count_out", "q_start", "pos", "slots", "ws", "free"):
        assert f(**{name: None}) == ARG, name
    assert f(page=24) == UNSUP and f(page=8) == UNSUP and f(T=1 << 31) == UNSUP
    assert f(ld=1 << 27, blocks=1 << 27) == UNSUP                    # 2^31 positions
    for name in ("new", "lens", "count", "lens_out", "count_out", "q_start", "pos", "table", "free"):
        assert f(**{name: ODD}) == ALIGN, name
    assert f(slots=ctypes.c_void_p(0x10004)) == ALIGN and f(ws=OFF8) == ALIGN
    assert f(bytes=255) == WS
    assert f(B=0) == OK


def test_norm_rope_append_refusals():
    two, three = i64(4096, 128), i64(4096, 2048, 128)
    f = caller(lib.think_norm_rope_append, q=FAKE, qs=two, k=FAKE, ks=two, v=FAKE, vs=two, T=4, Hq=4, Hkv=2, d=128, dtype=1,
               wq=FAKE, wk=FAKE, eps=1e-6, freq=FAKE, rot=128, nb=0, pos=FAKE, slots=FAKE, qo=FAKE, qos=two, kc=FAKE,
               kcs=three, vc=FAKE, vcs=three, pages=3, page=16)
    assert f(T=-1) == ARG and f(Hq=-1) == ARG and f(Hkv=-1) == ARG and f(dtype=2) == ARG and f(rot=-16) == ARG
    assert f(rot=144) == ARG and f(eps=-1.0) == ARG and f(eps=float("nan")) == ARG and f(eps=float("inf")) == ARG
    assert f(pages=0) == ARG and f(page=0) == ARG
    for name in ("q", "qs", "k", "ks", "v", "vs", "freq", "pos", "slots", "qo", "qos", "kc", "kcs", "vc", "vcs"):
        assert f(**{name: None}) == ARG, name
    assert f(d=64) == UNSUP and f(rot=24) == UNSUP and f(page=20) == UNSUP and f(Hq=70000) == UNSUP and f(T=1 << 31) == UNSUP
    for name in ("q", "k", "v", "qo", "kc", "vc", "wq", "wk"):
        assert f(**{name: OFF8}) == ALIGN, name
    for name in ("qs", "ks", "vs", "qos"):
        assert f(**{name: i64(4096, 132)}) == ALIGN and f(**{name: i64(-4096, 128)}) == ALIGN, name
    for name in ("kcs", "vcs"):
        assert f(**{name: i64(4096, 2048, 130)}) == ALIGN, name
    assert f(freq=ctypes.c_void_p(0x10004)) == ALIGN and f(pos=ODD) == ALIGN and f(slots=ctypes.c_void_p(0x10004)) == ALIGN
    assert f(T=0) == OK and f(Hq=0, Hkv=0) == OK


def test_paged_attn_refusals():
    two, three = i64(4096, 128), i64(4096, 2048, 128)
    ws = qdk.think_paged_attn_workspace_size(10, 4, 2)
    f = caller(lib.think_paged_attn, q=FAKE, qs=two, k=FAKE, ks=three, v=FAKE, vs=three, pages=3, page=16, table=FAKE, ld=8,
               blocks=8, q_start=FAKE, lens=FAKE, B=2, T=10, max_new=0, Hq=4, Hkv=2, d=128, dtype=1, scale=0.1, window=0,
               out=FAKE, os=two, ws=FAKE, bytes=ws)
    assert f(B=-1) == ARG and f(T=-1) == ARG and f(window=-1) == ARG and f(max_new=-1) == ARG and f(dtype=3) == ARG
    assert f(Hq=5) == ARG and f(Hq=1) == ARG and f(scale=float("nan")) == ARG and f(scale=float("inf")) == ARG
    assert f(pages=0) == ARG and f(page=0) == ARG and f(blocks=0) == ARG and f(ld=7) == ARG and f(table=None) == ARG
    for name in ("q", "qs", "k", "ks", "v", "vs", "q_start", "lens", "out", "os", "ws"):
        assert f(**{name: None}) == ARG, name
    assert f(d=64) == UNSUP and f(page=24) == UNSUP and f(blocks=1 << 27, ld=1 << 27) == UNSUP and f(T=1 << 31) == UNSUP
    assert f(Hq=2 * 4097) == UNSUP and f(T=1 << 28, Hq=64, Hkv=1) == UNSUP
    for name in ("q", "k", "v", "out", "ws"):
        assert f(**{name: OFF8}) == ALIGN, name
    assert f(q_start=ODD) == ALIGN and f(lens=ODD) == ALIGN and f(table=ODD) == ALIGN
    for name in ("qs", "os"):
        assert f(**{name: i64(4096, 132)}) == ALIGN, name
    for name in ("ks", "vs"):
        assert f(**{name: i64(4096, 2048, 130)}) == ALIGN, name
        assert f(**{name: i64(4096, 0, 128)}) == ARG and f(**{name: i64(0, 2048, 128)}) == ARG, name
        assert f(**{name: i64(1 << 40, 2048, 128)}) == UNSUP, name
    assert f(bytes=ws - 1) == WS
    assert f(B=0) == OK and f(T=0) == OK and f(Hkv=0) == OK


def test_paged_attn_refuses_pools_that_no_step_divides():
    ws = qdk.think_paged_attn_workspace_size(10, 4, 2)
    f = caller(lib.think_paged_attn, q=FAKE, qs=i64(4096, 128), k=FAKE, ks=i64(4096, 2048, 128), v=FAKE, vs=i64(4096, 2048, 128),
               pages=3, page=16, table=FAKE, ld=8, blocks=8, q_start=FAKE, lens=FAKE, B=2, T=10, max_new=0, Hq=4, Hkv=2, d=128,
               dtype=qdk.THINK_BF16, scale=0.1, window=0, out=FAKE, os=i64(4096, 128), ws=FAKE, bytes=ws)
    for name in ("ks", "vs"):
        assert f(**{name: i64(1 << 38, 24, 128)}) == UNSUP and f(**{name: i64(24, 1 << 38, 128)}) == UNSUP, name
        assert f(**{name: i64(4096, 2048, 1 << 36)}) == UNSUP, name  # eight rows apart by 2^40 bytes


def test_gather_refusals():
    three = i64(4096, 2048, 128)
    f = caller(lib.think_gather_pages, c=FAKE, cs=three, pages=3, page=16, table=FAKE, ld=8, blocks=8, lens=FAKE, B=2, Hkv=2,
               N=50, d=128, dtype=1, out=FAKE)
    assert f(B=-1) == ARG and f(Hkv=-1) == ARG and f(N=-1) == ARG and f(dtype=9) == ARG and f(pages=0) == ARG
    for name in ("c", "cs", "table", "lens", "out"):
        assert f(**{name: None}) == ARG, name
    assert f(d=96) == UNSUP and f(page=17) == UNSUP and f(B=70000) == UNSUP and f(N=(1 << 30) + 1) == UNSUP
    assert f(c=OFF8) == ALIGN and f(out=OFF8) == ALIGN and f(lens=ODD) == ALIGN and f(cs=i64(4096, 2048, 130)) == ALIGN
    assert f(B=0) == OK and f(N=0) == OK


def test_binding_refuses_what_is_not_on_a_gpu():
    t = torch.zeros(4, 2, 128)
    i = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: qdk.think_gather_pages(t, i, i, t),
                 lambda: qdk.think_paged_attn(t, t, t, i, i, i, t, t),
                 lambda: qdk.think_norm_rope_append(t, t, t, None, None, 1e-6, None, False, i, i, t, t, t),
                 lambda: qdk.think_extend_pages(i, i, i, i, i, 16, i, i, i, i, i, i),
                 lambda: qdk.think_gather_pages(None, i, i, t)):
        with pytest.raises(qdk.ThinkError) as e:
            call()
        assert e.value.code == ARG


def test_status_bits_are_distinct():
    bits = [v for k, v in vars(qdk).items() if k.startswith("THINK_DEVICE_")]
    assert len(bits) == len(set(bits)) == 7 and all(b & (b - 1) == 0 for b in bits)
