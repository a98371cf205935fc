"""Append and read of the paged 4-bit cache on both sides of the borders where a
warp takes other shares of the rows."""
import numpy as np
import pytest
import torch

import _kv4 as R
from test_gpu_kv4 import BF16, F16, F32

pytestmark = pytest.mark.gpu


# one row, AHEAD rows, all heads of a token a warp; 1, 2, 4 tokens
@pytest.mark.parametrize("D,group,dtype", [(128, 32, BF16), (128, 64, F32), (64, 32, F16), (64, 64, F32)])
@pytest.mark.parametrize("H,n", [(32, 127), (32, 128), (32, 256), (40, 2047), (40, 2048), (37, 300), (8, 511), (8, 1024),
                                 (3, 8191), (3, 8192), (3, 16384), (2, 16389)])
def test_shares(dkv_gpu, D, group, dtype, H, n):
    rng = np.random.default_rng(H + n + D)
    lens = [n - n // 3 - 1, 0, n // 3 + 1]
    t = R.Tables(lens, 48, n)
    cache = dkv_gpu.Kv4Cache(t.n_pages, H, head_dim=D, page_size=48, group=group)
    table, end = t.dev()
    starts, pad = R.starts_of(lens), 5
    k, v = (torch.from_numpy(rng.standard_normal((n + pad, H, D), np.float32)).to(dtype) for _ in range(2))
    cache.append(k.cuda(), v.cuda(), table, end, starts)
    out = tuple(torch.full((n + pad, H, D), -5.0, dtype=F32, device="cuda") for _ in range(2))
    cache.read(n + pad, table, end, starts, out=out)
    assert cache.device_status() == 0
    for y, x in zip(out, (k, v)):
        assert np.array_equal(y[:n].cpu().numpy(), R.held(x[:n].float().numpy(), group).astype(np.float32))
        assert bool((y[n:] == -5).all())
