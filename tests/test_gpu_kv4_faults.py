"""The paged 4-bit cache where something goes wrong: waits that run out, status
words, streams."""
import time

import numpy as np
import pytest
import torch

import _kv4 as R
from test_gpu_kv4 import BF16, F16, F32, fill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,group,dtype", [(128, 32, BF16), (64, 64, F16)])
def test_a_wait_that_runs_out(dkv_gpu, D, group, dtype):
    """Barriers armed for bytes that never come (all copies that are issued do
    land): the call returns, says so, and leaves the cache usable."""
    cache, table, end, _, _ = fill(dkv_gpu, [900, 0, 33, 4000], 2, D, group, 16, dtype, 1)
    q = torch.randn(4, 8, D, device="cuda", dtype=dtype)
    good = cache.decode_attn(q, 0.1, table, end)
    assert cache.device_status() == 0
    dkv_gpu.dkv_debug_set_fault(1)
    try:
        t0 = time.time()
        cache.decode_attn(q, 0.1, table, end)
        status = cache.device_status()
        took = time.time() - t0
    finally:
        dkv_gpu.dkv_debug_set_fault(0)
    assert status == dkv_gpu.DEV_TIMEOUT and took < 30
    assert torch.equal(cache.decode_attn(q, 0.1, table, end), good)
    assert cache.device_status() == 0
