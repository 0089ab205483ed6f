"""CPU: rows that a paged call would write several times to one place are refused."""
import ctypes

import pytest

qdk = pytest.importorskip("query_driven_key_b200")
lib = qdk.lib
P = ctypes.c_void_p(0x10000)  # never dereferenced: validation rejects first
ARG = qdk.THINK_ERR_INVALID_ARG


def i64(*x):
    return (ctypes.c_int64 * len(x))(*x)


def rope(qo=(512, 128), kc=(4096, 2048, 128), vc=(4096, 2048, 128), T=4, Hq=4, Hkv=2, pages=3):
    return lib.think_norm_rope_append(P, i64(512, 128), P, i64(512, 128), P, i64(512, 128), T, Hq, Hkv, 128, 1, None, None, 0.0,
                                      P, 128, 0, P, P, P, i64(*qo), P, i64(*kc), P, i64(*vc), pages, 16, None)


def attn(out=(512, 128), T=4, Hq=4, ws=1 << 40):
    return lib.think_paged_attn(P, i64(512, 128), P, i64(4096, 2048, 128), P, i64(4096, 2048, 128), 3, 16, P, 8, 8, P, P, 1, T, 0,
                                Hq, 2, 128, 1, 0.1, 0, P, i64(*out), P, ws, None)


def test_rotation_refuses_rows_in_one_place():
    for x in ((0, 128), (512, 0)):
        assert rope(qo=x) == ARG
    for x in ((0, 2048, 128), (4096, 0, 128), (4096, 2048, 0)):
        assert rope(kc=x) == ARG and rope(vc=x) == ARG


def test_attention_refuses_rows_in_one_place():
    assert attn(out=(0, 128)) == ARG and attn(out=(512, 0)) == ARG
    # a single token's stride is free: refused for its workspace only
    assert attn(out=(0, 128), T=1, ws=0) == qdk.THINK_ERR_WORKSPACE
