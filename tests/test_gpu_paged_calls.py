"""Calls of the paged cache that meet other threads, streams, refusals and extreme values, on the GPU."""
import threading

import pytest
import torch

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
