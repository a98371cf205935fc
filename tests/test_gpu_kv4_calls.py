"""The paged 4-bit cache's calls at their borders: quotients next to a tie, the
largest inputs, pools past 4 GB, refusals of the Python helper, calls that share
nothing, captured calls whose lengths change, and the bounds-checked build."""
import os
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import _kv4 as R
from test_gpu_kv4 import BF16, F16, F32, fill

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parents[1]


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_quotients_next_to_a_tie(dkv_gpu):
    """Every 7-bit scale of a binade, zero points from 0 to 15, and x within four
    fp32 steps of (k + 1/2) s: codes by numpy's correctly rounded division."""
    rng = np.random.default_rng(3)
    n, D, group = 8 * 4096, 64, 32
    m = rng.integers(64, 128, (n, 2))
    e = rng.integers(-18, 8, (n, 2))
    s = np.ldexp(m.astype(np.float64), e)
    zero = rng.integers(0, 16, (n, 2))
    k = rng.integers(-15, 16, (n, 2, group))
    x = ((k + 0.5) * s[..., None]).astype(np.float32)
    x = np.clip(x, (-zero * s)[..., None], ((15 - zero) * s)[..., None]).astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-4, 5, x.shape) * (x != 0)).astype(np.int32).view(np.float32)
    x[..., 0] = -zero * s                      # the extremes that make the scale about s
    x[..., 1] = (15 - zero) * s
    x = torch.from_numpy(x.reshape(n, 1, D))
    cache = dkv_gpu.Kv4Cache(n // 16, 1, head_dim=D, page_size=16, group=group)
    table = torch.arange(n // 16, dtype=torch.int32, device="cuda")[None]
    cache.append(x.cuda(), x.flip(0).contiguous().cuda(), table, i32(n))
    a, b = cache.read(n, table, i32(n), dtype=F32)
    want = R.held(x.numpy(), group)
    assert np.array_equal(a.cpu().numpy(), want.astype(np.float32))
    assert np.array_equal(b.cpu().numpy(), want[::-1].astype(np.float32))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_inputs_past_the_range(dkv_gpu, dtype):
    """NaN, infinities and values past 32768 in some blocks, others beside them in
    the same warps as they are."""
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.normal(size=(37, 3, 128)).astype(np.float32))
    x[3, 1, 5], x[9, 0, 64], x[9, 2, 100] = float("nan"), float("inf"), -float("inf")
    x[20, 1, 33], x[21, 1, 34] = 40000.0, -60000.0
    x[30] = float("nan")
    x = x.to(dtype)
    cache = dkv_gpu.Kv4Cache(3, 3, page_size=16)
    table = i32(0, 1, 2)[None]
    cache.append(x.cuda(), x.cuda(), table, i32(37))
    for y in cache.read(37, table, i32(37), dtype=F32):
        assert np.array_equal(y.cpu().numpy(), R.held(x.float().numpy(), 32).astype(np.float32))


def test_pool_past_4_gigabytes(dkv_gpu):
    H, page = 8, 64
    n_pages = 70000
    cache = dkv_gpu.Kv4Cache(n_pages, H, page_size=page)
    assert cache.pool.numel() > 5 * 2 ** 30 - 2 ** 28
    rng = np.random.default_rng(5)
    n = 3 * page - 7
    k, v = (R.make_kv(rng, n, H, 128, F16) for _ in range(2))
    table = i32(n_pages - 1, 3, n_pages - 2)[None]
    cache.append(k.cuda(), v.cuda(), table, i32(n))
    for y, x in zip(cache.read(n, table, i32(n), dtype=F32), (k, v)):
        assert np.array_equal(y.cpu().numpy(), R.held(x.float().numpy(), 32).astype(np.float32))
    q = torch.randn(n, 2 * H, 128, device="cuda", dtype=F16)
    a = cache.prompt_attn(q, 0.09, table, i32(n))
    b = cache.decode_attn(q[-1:], 0.09, table, i32(n))
    for out, rows in ((a[-1:], [n - 1]), (b, [n - 1]), (a[100:101], [100])):
        want = [R.attention(q[rows, h].double().cpu().numpy(), R.held(k.float().numpy()[:, h // 2], 32),
                            R.held(v.float().numpy()[:, h // 2], 32), R.step(k.float().numpy()[:, h // 2], 32),
                            R.step(v.float().numpy()[:, h // 2], 32), np.array(rows), 0.09, 0) for h in range(2 * H)]
        R.check(out, None, want, F16)
    assert cache.device_status() == 0


def test_refusals_of_the_helper(dkv_gpu):
    d = dkv_gpu
    cache, table, end, _, _ = fill(d, [40, 20], 2, 64, 32, 16, F16, 1)
    k = torch.randn(2, 2, 64, device="cuda", dtype=F16)
    q = torch.randn(2, 4, 64, device="cuda", dtype=F16)
    for bad in (dict(block_table=table.long()), dict(block_table=table[0]), dict(block_table=table[:1]),
                dict(block_table=table.cpu()), dict(seq_lens=end.float()), dict(seq_lens=end.cpu()),
                dict(seq_lens=end[:1]), dict(block_table=table.t().contiguous().t())):
        kw = dict(dict(block_table=table, seq_lens=end), **bad)
        for call in (lambda: cache.append(k, k, **kw), lambda: cache.read(2, **kw),
                     lambda: cache.decode_attn(q, 0.1, **kw), lambda: cache.prompt_attn(q, 0.1, **kw)):
            with pytest.raises(ValueError):
                call()
    for starts in (i32(0, 1), i32(0, 1, 2, 2), i32(0, 1, 2).long(), torch.zeros(3, dtype=torch.int32)):
        for call in (lambda: cache.append(k, k, table, end, starts), lambda: cache.read(2, table, end, starts),
                     lambda: cache.prompt_attn(q, 0.1, table, end, starts)):
            with pytest.raises(ValueError):
                call()
    for x in (k.cpu(), k[0], k[:, :1], k[..., :32], k.double(), k.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            cache.append(x, x, table, end)
    with pytest.raises(ValueError):
        cache.append(k, k.float(), table, end)
    for x in (q.cpu(), q[0], q[..., :32], q.double()):
        for call in (cache.decode_attn, cache.prompt_attn):
            with pytest.raises(ValueError):
                call(x, 0.1, table, end)
    with pytest.raises(ValueError):
        cache.decode_attn(q[:1], 0.1, table, end)
    for out in (torch.empty_like(q).float(), torch.empty(2, 4, 128, device="cuda", dtype=F16)[..., :64],
                torch.empty(2, 4, 64, dtype=F16)):
        for call in (cache.decode_attn, cache.prompt_attn):
            with pytest.raises(ValueError):
                call(q, 0.1, table, end, out=out)
    with pytest.raises(ValueError):
        cache.read(2, table, end, out=(k, k.float()))
    for scale, window, x in ((0.0, 0, q), (float("nan"), 0, q), (0.1, -1, q), (0.1, 0, q[:, :3]), (0.1, 0, q.float())):
        for call in (cache.decode_attn, cache.prompt_attn):
            with pytest.raises(d.DkvError):
                call(x, scale, table, end, window=window)
    with pytest.raises(d.DkvError):
        cache.decode_attn(torch.randn(2, 17, 4, 64, device="cuda", dtype=F16), 0.1, table, end)
    with pytest.raises(d.DkvError):
        d.Kv4Cache(4, 2, head_dim=96)
    # nothing to do is not an error
    cache.append(k[:0], k[:0], table, end)
    assert cache.read(0, table, end)[0].shape == (0, 2, 64)
    assert cache.prompt_attn(q[:0], 0.1, table, end).shape == (0, 4, 64)
    assert cache.device_status() == 0


def test_queries_in_any_layout(dkv_gpu):
    """Strided rows and heads, an expanded batch, batches of several queries
    whose rows have no single stride."""
    cache, table, end, _, _ = fill(dkv_gpu, [40, 20], 2, 128, 32, 16, F16, 1)
    q = torch.randn(2, 3, 4, 128, device="cuda", dtype=F16)
    want = cache.decode_attn(q, 0.1, table, end)
    wide = torch.zeros(2, 5, 8, 160, device="cuda", dtype=F16)
    wide[:, :3, ::2, 16:144] = q
    assert torch.equal(cache.decode_attn(wide[:, :3, ::2, 16:144], 0.1, table, end), want)
    heads_first = q.reshape(6, 4, 128).transpose(0, 1).contiguous().transpose(0, 1)
    a = cache.prompt_attn(q.reshape(6, 4, 128), 0.1, table, end)
    assert torch.equal(cache.prompt_attn(heads_first, 0.1, table, end), a)
    one = q[:1, :1].expand(2, 3, 4, 128)
    assert torch.equal(cache.decode_attn(one, 0.1, table, end), cache.decode_attn(one.contiguous(), 0.1, table, end))


@pytest.mark.parametrize("window", [2 ** 30, 2 ** 30 + 1, 2 ** 31 - 16, 2 ** 31 - 1])
def test_windows_past_every_position(dkv_gpu, window):
    """Sequences shorter than the queries among them."""
    cache, table, end, _, _ = fill(dkv_gpu, [400, 1, 0, 9], 2, 128, 32, 16, F16, 1)
    q = torch.randn(4, 16, 4, 128, device="cuda", dtype=F16)
    assert torch.equal(cache.decode_attn(q, 0.1, table, end, window=window), cache.decode_attn(q, 0.1, table, end))
    starts, rows = i32(0, 300, 301, 301, 310), torch.randn(310, 4, 128, device="cuda", dtype=F16)
    assert torch.equal(cache.prompt_attn(rows, 0.1, table, end, starts, window=window),
                       cache.prompt_attn(rows, 0.1, table, end, starts))
    assert cache.device_status() == 0


def test_calls_repeat_bit_for_bit(dkv_gpu):
    cache, table, end, _, _ = fill(dkv_gpu, [5000, 300, 0, 77], 2, 128, 32, 64, BF16, 1)
    q = torch.randn(4 * 70, 8, 128, device="cuda", dtype=BF16)
    starts = i32(0, 200, 203, 203, 280)
    end[3] = 77
    for call in (lambda: cache.prompt_attn(q, 0.1, table, end, starts, return_lse=True),
                 lambda: cache.decode_attn(q[:4], 0.1, table, end, return_lse=True)):
        first = call()
        for _ in range(5):
            for x, y in zip(first, call()):
                assert torch.equal(x, y)


def test_two_graphs_and_an_eager_stream(dkv_gpu):
    """Captured prompt and decode calls on pools of their own, replayed at once
    with an eager call on a third stream; the lengths change between replays."""
    sets = []
    for seed in range(3):
        lens = [3000 + seed, 70]
        cache, table, end, _, _ = fill(dkv_gpu, lens, 2, 128, 32, 64, F16, seed)
        q = torch.randn(128, 8, 128, device="cuda", dtype=F16)
        sets.append((cache, table, end, q))

    def both(cache, table, end, q):
        return (cache.prompt_attn(q, 0.09, table, end, starts), cache.decode_attn(q[:2], 0.09, table, end))

    starts = i32(0, 100, 128)
    graphs = []
    for s in sets[:2]:
        both(*s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = both(*s)
        graphs.append((g, y))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for ends in ((3000, 70), (1500, 28), (130, 64)):
        for s in sets:
            s[2].copy_(torch.tensor(ends, dtype=torch.int32))
        want = [both(*s) for s in sets]
        torch.cuda.synchronize()
        got = []
        for _ in range(4):
            for i, st in enumerate(streams):
                with torch.cuda.stream(st):
                    if i < 2:
                        graphs[i][0].replay()
                    else:
                        got.append(both(*sets[2]))
        torch.cuda.synchronize()
        for i in range(2):
            for x, y in zip(graphs[i][1], want[i]):
                assert torch.equal(x, y)
        for z in got:
            for x, y in zip(z, want[2]):
                assert torch.equal(x, y)
        assert all(s[0].device_status() == 0 for s in sets)


def test_another_stream_by_handle(dkv_gpu):
    cache, table, end, _, _ = fill(dkv_gpu, [300, 20], 2, 64, 64, 16, BF16, 1)
    q = torch.randn(2, 4, 64, device="cuda", dtype=BF16)
    want = cache.decode_attn(q, 0.1, table, end)
    k, v = cache.read(2, table, end, dtype=F32)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for s in (st, st.cuda_stream):
        a = cache.decode_attn(q, 0.1, table, end, stream=s)
        b = cache.prompt_attn(q, 0.1, table, end, stream=s)
        c = cache.read(2, table, end, dtype=F32, stream=s)
        assert cache.device_status(stream=s) == 0
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.allclose(b.float(), want.float(), rtol=2 ** -6, atol=2e-3)
        assert torch.equal(c[0], k) and torch.equal(c[1], v)


def test_on_the_checked_build():
    """The cache's tests again with every computed range tested against its
    buffer (see test_gpu_checked.py)."""
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        *[str(ROOT / "tests" / f) for f in ("test_gpu_kv4.py", "test_gpu_kv4_prompt.py")]],
                       cwd=ROOT, env=dict(os.environ, DKV_LIBRARY="checked"), capture_output=True, text=True,
                       timeout=1500)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
