"""The paged 4-bit cache at the largest counts it takes, and calls whose very
first run is captured into a graph."""
import math
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import _kv4 as R
from test_gpu_kv4 import BF16, F16, F32, decode_case, fill
from test_gpu_kv4_prompt import prompt_case

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parents[1]


@pytest.mark.parametrize("page", [128, 144, 256, 4096, 65536])
@pytest.mark.parametrize("D,group,dtype", [(128, 32, F16), (64, 64, BF16)])
def test_large_pages(dkv_gpu, page, D, group, dtype):
    lens, new = [700, 0, 150, 129], [260, 0, 150, 1]
    decode_case(dkv_gpu, lens, 2, 3, D, group, page, dtype, 2, 0, seed=page)
    decode_case(dkv_gpu, lens, 2, 3, D, group, page, dtype, 1, 131, seed=page)
    prompt_case(dkv_gpu, lens, new, 2, 3, D, group, page, dtype, seed=page, every=9)
    prompt_case(dkv_gpu, lens, new, 2, 3, D, group, page, dtype, window=131, seed=page, every=9)


@pytest.mark.parametrize("G", [40, 300, 1024])
def test_many_query_heads_of_one_kv_head(dkv_gpu, G):
    decode_case(dkv_gpu, [130, 3, 0], 1, G, 64, 32, 16, BF16, 2, 0, seed=G)
    prompt_case(dkv_gpu, [400, 33, 5], [9, 33, 0], 1, G, 64, 32, 16, BF16, seed=G, pad=1, every=4)
    prompt_case(dkv_gpu, [400, 33, 5], [9, 33, 0], 1, G, 64, 32, 16, F16, window=50, seed=G, every=4)


def test_sixteen_thousand_sequences(dkv_gpu):
    B, H, G, D, page = 16384, 2, 2, 64, 16
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 4, B).astype(np.int32)
    n = int(lens.sum())
    table = torch.from_numpy(rng.permutation(B).astype(np.int32)[:, None]).cuda()
    end = torch.from_numpy(lens).cuda()
    cache = dkv_gpu.Kv4Cache(B, H, head_dim=D, page_size=page)
    k, v = (R.make_kv(rng, n, H, D, F16).cuda() for _ in range(2))
    starts = R.starts_of(lens)
    cache.append(k, v, table, end, starts)
    hk, hv = cache.read(n, table, end, starts, dtype=F32)
    for x, y in ((k, hk), (v, hv)):
        assert np.array_equal(y.cpu().numpy(), R.held(x.float().cpu().numpy(), 32).astype(np.float32))
    # every sequence's last position asks; the prompt call has the same rows
    has = torch.from_numpy(lens > 0).cuda()
    q = torch.randn(B, H * G, D, device="cuda", dtype=F16)
    one = torch.from_numpy(np.concatenate([[0], np.cumsum(lens > 0)]).astype(np.int32)).cuda()
    got = [(*cache.decode_attn(q, 0.1, table, end, return_lse=True), False)]
    got = [(y[has], l[has], e) for y, l, e in got] + \
        [(*cache.prompt_attn(q[has], 0.1, table, end, one, return_lse=True), True)]
    assert cache.device_status() == 0
    last = (torch.cumsum(end, 0)[has] - 1).long()
    idx = last[:, None] - torch.arange(3, device="cuda")
    seen = torch.arange(3, device="cuda") < end[has][:, None]
    idx = idx.clamp_min(0)
    kk, vv = (x.double()[idx].repeat_interleave(G, 2) for x in (hk, hv))          # [seqs, 3, Hq, D]
    x = torch.einsum("bhd,bjhd->bhj", q[has].double(), kk) * 0.1
    x = x.masked_fill(~seen[:, None], -math.inf)
    p = torch.softmax(x, -1)
    want, lse = torch.einsum("bhj,bjhd->bhd", p, vv), torch.logsumexp(x, -1)
    # weights rounded to fp16 once (2^-11), scores to 2^-18, the output (2^-11); the
    # decode's truncated sums: 2 (34 + 2) 2^-23 of up to 15 scales, which are below 2
    # for values up to 15
    a = torch.einsum("bhj,bjhd->bhd", p, vv.abs())
    for y, l, exact in got:
        tol = 2.0 ** -10 * a + 2.0 ** -11 * want.abs() + 2.0 ** -25 + (0 if exact else 72 * 30 * 2.0 ** -23)
        assert bool(((y.double() - want).abs() <= tol).all())
        assert bool(((l.double() - lse).abs() <= 2.0 ** -14).all())


@pytest.mark.parametrize("D,group", [(64, 64), (128, 32)])
def test_four_thousand_heads(dkv_gpu, D, group):
    H, n = 4096, 21
    rng = np.random.default_rng(2)
    cache = dkv_gpu.Kv4Cache(3, H, head_dim=D, page_size=16, group=group)
    table, end = torch.tensor([[2, 0]], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda()
    k, v = (R.make_kv(rng, n, H, D, F16).cuda() for _ in range(2))
    cache.append(k, v, table, end)
    hk, hv = cache.read(n, table, end, dtype=F32)
    for x, y in ((k, hk), (v, hv)):
        assert np.array_equal(y.cpu().numpy(), R.held(x.float().cpu().numpy(), group).astype(np.float32))
    q = torch.randn(n, H, D, device="cuda", dtype=F16)
    for out, at in ((cache.decode_attn(q[-1:], 0.1, table, end), [n - 1]),
                    (cache.prompt_attn(q, 0.1, table, end)[[3, n - 1]], [3, n - 1])):
        for h in (0, 1, 2047, 4095):
            z = [x[:, h].float().cpu().numpy() for x in (k, v)]
            want = [R.attention(q[at, h].double().cpu().numpy(), R.held(z[0], group), R.held(z[1], group),
                                R.step(z[0], group), R.step(z[1], group), np.array(at), 0.1, 0)]
            R.check(out[:, h:h + 1], None, want, F16)
    assert cache.device_status() == 0


_FIRST = r"""
import sys
sys.path.insert(0, ".")
import torch
import delta_quantized_kv_b200 as d
H, D = 2, 128
cache = d.Kv4Cache(8, H, page_size=16)
table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
end = torch.tensor([100], dtype=torch.int32, device="cuda")
x = torch.randn(100, 8 * H, D, device="cuda", dtype=torch.float16)
torch.cuda.synchronize()

def step():
    cache.append(x[:, :H], x[:, H:2 * H], table, end)
    return (cache.prompt_attn(x[:, 2 * H:6 * H], 0.1, table, end),
            cache.decode_attn(x[-1:, 2 * H:6 * H], 0.1, table, end), *cache.read(100, table, end))

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = step()
g.replay()
z = step()
torch.cuda.synchronize()
print("SAME", all(bool(torch.equal(a, b)) for a, b in zip(y, z)), cache.device_status())
"""


def test_the_first_calls_of_a_process_are_captured():
    r = subprocess.run([sys.executable, "-c", _FIRST], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.stdout + r.stderr)[-2000:]
    assert "SAME True 0" in r.stdout
