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


def attention_of(ks, vs, q, group, pos, scale, window):
    G = q.shape[1] // ks.shape[1]
    return [R.attention(q[:, h].double().cpu().numpy(), R.held(ks[:, h // G], group), R.held(vs[:, h // G], group),
                        R.step(ks[:, h // G], group), R.step(vs[:, h // G], group), pos, scale, window)
            for h in range(q.shape[1])]


@pytest.mark.parametrize("D,group", [(128, 32), (128, 64), (64, 32), (64, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("nq,window", [(1, 0), (1, 13), (3, 0), (3, 37)])
def test_values_that_no_query_sees_leave_every_bit(dkv_gpu, D, group, dtype, nq, window):
    """Huge values behind the lengths (a recycled page's) and before the windows,
    small ones where the queries look: the bits of a cache that holds zeros there."""
    H, G, page, lens = 2, 3, 32, [20, 45, 71, 8, 64]
    rng = np.random.default_rng(D + group + nq + window)
    t = R.Tables(lens, page, 3)
    table, end = t.dev()
    full = [-(-n // page) * page for n in lens]
    first = np.concatenate([[0], np.cumsum(full)])
    k = rng.normal(size=(first[-1], H, D)).astype(np.float32)
    v = (rng.normal(size=(first[-1], H, D)) * 1e-2).astype(np.float32)
    seen = np.zeros(first[-1], bool)
    for b, n in enumerate(lens):
        lo = max(0, n - nq + 1 - window) if window else 0
        seen[first[b] + lo:first[b] + n] = True
    q = torch.from_numpy(rng.normal(size=(len(lens), nq, H * G, D)) * 3).to(dtype).cuda()
    scale, got = 1 / D ** 0.5, []
    for far in (0.0, 3e4):
        x = np.where(seen[:, None, None], v, np.where(rng.random(v.shape) < 0.5, far, -far)).astype(np.float32)
        cache = dkv_gpu.Kv4Cache(t.n_pages, H, head_dim=D, page_size=page, group=group)
        cache.append(torch.from_numpy(k).to(dtype).cuda(), torch.from_numpy(x).to(dtype).cuda(), table,
                     torch.tensor(full, dtype=torch.int32).cuda(), R.starts_of(full))
        got.append(cache.decode_attn(q, scale, table, end, window=window, return_lse=True))
        assert cache.device_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
    kk, vv = (torch.from_numpy(y).to(dtype).float().numpy() for y in (k, v))
    for b, n in enumerate(lens):
        rows = slice(first[b], first[b] + n)
        want = attention_of(kk[rows], vv[rows], q[b], group, n - nq + np.arange(nq), scale, window)
        R.check(got[1][0][b], got[1][1][b], want, dtype)


def test_a_cache_made_on_another_stream(dkv_gpu):
    """Its pages are zero although the current stream has a write to a block
    of their size, given back already, still before it."""
    H, page, n_pages = 8, 64, 400
    size = n_pages * dkv_gpu.dkv_kv4_page_bytes(dkv_gpu.dkv_kv4_desc(H, 128, 32, page))
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        x = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(200_000_000)                 # about 0.1 s
        x.fill_(255)
        del x
        cache = dkv_gpu.Kv4Cache(n_pages, H, page_size=page, stream=stream)
        torch.cuda.synchronize()
        base = cache.c.base - cache.pool.data_ptr()
        assert not bool(cache.pool[base:base + size].any())
        assert cache.device_status(stream=stream) == 0
        del cache


@pytest.mark.parametrize("paged", [False, True])
def test_a_delta_cache_made_on_another_stream(dkv_gpu, paged):
    kw = dict(page_groups=1) if paged else {}
    plain = dkv_gpu.Cache(2, 2, 64, **kw)
    k, v = torch.randn(2, 2, 2, 50, 128, device="cuda", dtype=F16)
    q = torch.randn(2, 4, 128, device="cuda", dtype=F16)
    plain.encode(k, v)
    want = plain.decode_attn(q, 0.1)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        x = torch.empty(plain.buf.numel(), dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(200_000_000)                 # about 0.1 s
        x.fill_(255)
        del x
        cache = dkv_gpu.Cache(2, 2, 64, stream=stream, **kw)
        cache.encode(k, v, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(cache.decode_attn(q, 0.1), want)
        assert cache.device_status() == 0


def test_every_fault_is_reported(dkv_gpu):
    """Calls with bad lengths and bad pages on one stream, status reads on
    another meanwhile: no report is lost."""
    d = dkv_gpu
    cache, table, end, _, _ = fill(d, [40, 20], 1, 64, 32, 16, F16, 1)
    q = torch.randn(2, 1, 64, device="cuda", dtype=F16)
    bad_page, bad_len = table.clone(), end.clone()
    bad_page[0, 0], bad_len[1] = 10 ** 6, -1
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    rng = np.random.default_rng(1)
    for i in range(100):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(int(rng.integers(0, 100_000)))
            cache.decode_attn(q, 0.1, bad_page, end)
            torch.cuda._sleep(int(rng.integers(0, 50_000)))
            cache.decode_attn(q, 0.1, table, bad_len)
            done.record()
        got, last = 0, False
        while not last:
            last = done.query()
            got |= cache.device_status()
        assert got == d.DEV_BAD_PAGE | d.DEV_BAD_SEQLEN, i
    assert cache.device_status() == 0 and int(cache.status.item()) == 0


def test_rows_before_the_first_sequence_are_padding(dkv_gpu):
    """starts[0] > 0: such rows are passed over, and are no fault."""
    cache, table, end, _, _ = fill(dkv_gpu, [40, 20], 2, 64, 32, 16, F16, 1)
    k = torch.randn(12, 2, 64, device="cuda", dtype=F16)
    starts = torch.tensor([4, 7, 10], dtype=torch.int32, device="cuda")
    cache.append(k, k, table, end, starts)
    assert cache.device_status() == 0
    out = tuple(torch.full((12, 2, 64), -5.0, device="cuda", dtype=F32) for _ in range(2))
    cache.read(12, table, end, starts, out=out)
    assert cache.device_status() == 0
    for y in out:
        assert np.array_equal(y[4:10].cpu().numpy(), R.held(k[4:10].float().cpu().numpy(), 32).astype(np.float32))
        assert bool((y[:4] == -5).all()) and bool((y[10:] == -5).all())
    q = torch.randn(12, 4, 64, device="cuda", dtype=F16)
    a, b = torch.full_like(q, -5), torch.full_like(q[4:10], -5)
    cache.prompt_attn(q, 0.1, table, end, starts, out=a)
    cache.prompt_attn(q[4:10], 0.1, table, end, starts - 4, out=b)
    assert torch.equal(a[4:10], b) and bool((a[:4] == -5).all()) and bool((a[10:] == -5).all())
    assert cache.device_status() == 0


@pytest.mark.parametrize("dtype,scale,gain", [(F16, 1e-44, 1.0), (BF16, 1e-44, 1.0), (BF16, 1e-10, 1e-34),
                                              (F16, 1e-30, 1e-4)])
def test_scores_too_small_for_a_float(dkv_gpu, dtype, scale, gain):
    """All weights are the same: the mean of the values seen."""
    lens, new, H, D = [300, 40], [150, 9], 1, 64
    cache, table, end, ks, vs = fill(dkv_gpu, lens, H, D, 32, 16, dtype, 3)
    q = (torch.randn(sum(new), 2, D, device="cuda") * gain).to(dtype)
    out, lse = cache.prompt_attn(q, scale, table, end, R.starts_of(new), return_lse=True)
    last = torch.stack([q[new[0] - 1], q[-1]])
    one, lse_one = cache.decode_attn(last, scale, table, end, return_lse=True)
    assert cache.device_status() == 0
    row = 0
    for b, n in enumerate(lens):
        pos = n - new[b] + np.arange(new[b])
        rows = slice(row, row + new[b])
        R.check(out[rows], lse[rows], attention_of(ks[b], vs[b], q[rows], 32, pos, scale, 0), dtype, exact_values=True)
        R.check(one[b:b + 1], lse_one[b:b + 1], attention_of(ks[b], vs[b], last[b:b + 1], 32, pos[-1:], scale, 0), dtype)
        row += new[b]
