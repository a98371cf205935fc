"""The paged 4-bit cache on the GPU: what is written and read back against the
block rule in numpy, and decode attention against float64."""
import math

import numpy as np
import pytest
import torch

import _kv4 as R

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def fill(dkv, lens, H, D, group, page, dtype, seed, spare=2):
    """A cache holding sequences of the given lengths, and the inputs by sequence."""
    rng = np.random.default_rng(seed)
    t = R.Tables(lens, page, seed, spare)
    cache = dkv.Kv4Cache(t.n_pages, H, head_dim=D, page_size=page, group=group)
    table, end = t.dev()
    n = int(sum(lens))
    k, v = (R.make_kv(rng, max(n, 1), H, D, dtype)[:n] for _ in range(2))
    cache.append(k.cuda(), v.cuda(), table, end, R.starts_of(lens))
    first = np.concatenate([[0], np.cumsum(lens)])
    rows = [slice(first[b], first[b + 1]) for b in range(len(lens))]
    return cache, table, end, [k[r].float().numpy() for r in rows], [v[r].float().numpy() for r in rows]


@pytest.mark.parametrize("D,group", [(128, 32), (128, 64), (64, 32), (64, 64)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("page,H", [(16, 1), (48, 5), (64, 8)])
def test_append_and_read_are_the_block_rule(dkv_gpu, D, group, dtype, page, H):
    lens, new = [1, 40, 0, 129, 17, 16, 33], [1, 7, 0, 100, 17, 1, 0]
    rng = np.random.default_rng(D + page)
    t = R.Tables(lens, page, 3)
    cache = dkv_gpu.Kv4Cache(t.n_pages, H, head_dim=D, page_size=page, group=group)
    table, end = t.dev()
    first = [n - c for n, c in zip(lens, new)]
    # behind contexts written by an earlier call; views of one fused projection; padding rows
    ctx_k, ctx_v = (R.make_kv(rng, sum(first), H, D, dtype) for _ in range(2))
    cache.append(ctx_k.cuda(), ctx_v.cuda(), table,
                 torch.tensor(first, dtype=torch.int32).cuda(), R.starts_of(first))
    pad = 3
    n = sum(new)
    fused = torch.full((n + pad, 3 * H * D), 7.0, dtype=dtype)
    k, v = (R.make_kv(rng, n, H, D, dtype) for _ in range(2))
    fused[:n, H * D:2 * H * D] = k.view(n, -1)
    fused[:n, 2 * H * D:] = v.view(n, -1)
    fused = fused.cuda()
    kk, vv = (fused[:, i * H * D:(i + 1) * H * D].view(n + pad, H, D) for i in (1, 2))
    starts = R.starts_of(new)
    cache.append(kk, vv, table, end, starts)
    assert cache.device_status() == 0

    want = [R.held(x.float().numpy(), group) for x in (k, v)]
    for dt in (F16, F32, BF16):
        out = tuple(torch.full((n + pad, H, D), -5.0, dtype=dt, device="cuda") for _ in range(2))
        cache.read(n + pad, table, end, starts, out=out)
        for x, w in zip(out, want):
            assert torch.equal(x[:n].cpu(), torch.from_numpy(w).to(dt)), dt
            assert bool((x[n:] == -5).all())
    # the contexts are still there
    x = cache.read(sum(first), table, torch.tensor(first, dtype=torch.int32).cuda(),
                   R.starts_of(first))
    for y, w in zip(x, (ctx_k, ctx_v)):
        assert torch.equal(y.cpu().double(), torch.from_numpy(R.held(w.float().numpy(), group)))


@pytest.mark.parametrize("D,group", [(128, 32), (64, 64)])
def test_block_rule_corners(dkv_gpu, D, group):
    """NaN, infinities, all-zero and one-sided blocks, tiny and huge ranges, ties."""
    rng = np.random.default_rng(5)
    x = rng.normal(size=(64, 1, D)).astype(np.float32)
    x[0] = 0
    x[1, 0, 3], x[2, 0, 5], x[3, 0, 7] = np.nan, np.inf, -np.inf
    x[4] = np.nan
    x[5], x[6] = np.abs(x[5]) + 1, -np.abs(x[6]) - 1
    for i, p in enumerate(range(-150, 20, 5)):
        x[8 + i] = np.ldexp(x[8 + i], p).astype(np.float32)
    x[50] = 1e-45
    x[51] = 3.0e38 * np.sign(x[51])
    x[52] = np.arange(D) % 16 - 7.5
    x[53] = (np.arange(D) % 31 - 15) * 0.5
    x[54] = 65504.0
    x[55, 0, :] = 2.0 ** -14 * 15
    x[56, 0, :] = np.float32(2.0 ** -14 * 15) * np.float32(1 - 2.0 ** -20)
    n = len(x)
    t = R.Tables([n], 16, 1)
    cache = dkv_gpu.Kv4Cache(t.n_pages, 1, head_dim=D, page_size=16, group=group)
    table, end = t.dev()
    k = torch.from_numpy(x).cuda()
    cache.append(k, -k, table, end)
    a, b = cache.read(n, table, end, dtype=F32)
    assert np.array_equal(a.cpu().numpy(), R.held(x, group).astype(np.float32))
    assert np.array_equal(b.cpu().numpy(), R.held(-x, group).astype(np.float32))
    assert bool(torch.isfinite(a).all())
    # within half a step of what was given.  A block takes s = 0 only where its
    # range / 15 rounds to 0 in fp32, that is range / 15 <= 2^-150: then every
    # |x| <= 15 * 2^-150 < 2^-146
    y = np.clip(np.nan_to_num(x.astype(np.float64), nan=0.0, posinf=32768, neginf=-32768), -32768, 32768)
    s = R.quantise(x, group)[2].repeat(group, -1)
    assert np.all(np.abs(a.cpu().numpy() - y) <= 0.5 * s * (1 + 2.0 ** -18) + 2.0 ** -146 * (s == 0))


def decode_case(dkv, lens, H, G, D, group, page, dtype, nq, window, seed=0, scale=None, gain=1.0,
                strided=True):
    cache, table, end, ks, vs = fill(dkv, lens, H, D, group, page, dtype, seed)
    rng = np.random.default_rng(seed + 1)
    B, scale = len(lens), 1 / math.sqrt(D) if scale is None else scale
    fused = torch.from_numpy(rng.normal(size=(B * nq, (G + 1) * H, D)) * gain).to(dtype).cuda()
    q = fused[:, :G * H] if strided else fused[:, :G * H].contiguous()
    q = q.unflatten(0, (B, nq)) if nq > 1 else q
    out, lse = cache.decode_attn(q, scale, table, end, window=window, return_lse=True)
    assert cache.device_status() == 0
    assert out.shape == q.shape and out.dtype == dtype
    qf = q.reshape(B, nq, G * H, D).double().cpu().numpy()
    for b, n in enumerate(lens):
        want = []
        for h in range(G * H):
            k, v = ks[b][:, h // G], vs[b][:, h // G]
            want.append(R.attention(qf[b, :, h], R.held(k, group), R.held(v, group),
                                    R.step(k, group), R.step(v, group),
                                    n - nq + np.arange(nq), scale, window))
        R.check(out.reshape(B, nq, G * H, D)[b], lse.reshape(B, nq, G * H)[b], want, dtype)


RAGGED = [1, 300, 0, 16, 17, 31, 32, 33, 1000, 15]


@pytest.mark.parametrize("D,group", [(128, 32), (128, 64), (64, 32), (64, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("page,H,G", [(16, 1, 1), (64, 2, 4), (48, 3, 7)])
def test_decode_ragged(dkv_gpu, D, group, dtype, page, H, G):
    decode_case(dkv_gpu, RAGGED, H, G, D, group, page, dtype, 1, 0, seed=D + page)


@pytest.mark.parametrize("nq,G", [(2, 4), (3, 8), (5, 3), (16, 1), (4, 12)])
@pytest.mark.parametrize("window", [0, 20])
def test_decode_several_queries(dkv_gpu, nq, G, window):
    """Causal among the newest positions; sequences shorter than the queries
    leave the first of them without a position."""
    decode_case(dkv_gpu, [40, 1, 0, 3, 16, 333], 2, G, 128, 32, 32, F16, nq, window, seed=nq)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 100000])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_decode_window(dkv_gpu, window, dtype):
    decode_case(dkv_gpu, [5, 200, 16, 1025, 0], 2, 5, 64, 32, 16, dtype, 1, window, seed=window)


def test_decode_long_split_over_the_grid(dkv_gpu):
    decode_case(dkv_gpu, [70001, 3, 9000], 2, 8, 128, 32, 64, F16, 1, 0, seed=9)


def test_decode_many_sequences(dkv_gpu):
    decode_case(dkv_gpu, [(7 * i) % 90 for i in range(150)], 4, 2, 64, 64, 16, BF16, 1, 0, seed=10)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("gain", [1e-4, 30.0, 1000.0])
def test_decode_query_magnitudes(dkv_gpu, dtype, gain):
    """From a flat softmax to one position taking all."""
    decode_case(dkv_gpu, [500, 33], 1, 4, 128, 32, 64, dtype, 1, 0, seed=3, gain=gain)


@pytest.mark.parametrize("size", [2.0 ** -12, 1.0, 4000.0])
def test_decode_value_magnitudes(dkv_gpu, size):
    """V far from 1 (its scales move the weights' power of two), growing along
    the sequence so that the bound is passed in mid-run."""
    D, H, n, group = 128, 1, 600, 32
    rng = np.random.default_rng(8)
    k = torch.from_numpy(rng.normal(size=(n, H, D))).to(F16)
    v = torch.from_numpy(rng.normal(size=(n, H, D)) * size * np.linspace(0.01, 2, n)[:, None, None]).to(F16)
    t = R.Tables([n], 64, 2)
    cache = dkv_gpu.Kv4Cache(t.n_pages, H, head_dim=D, group=group)
    table, end = t.dev()
    cache.append(k.cuda(), v.cuda(), table, end)
    q = torch.from_numpy(rng.normal(size=(1, 4, D))).to(F16)
    out, lse = cache.decode_attn(q.cuda(), 0.1, table, end, return_lse=True)
    kf, vf = k[:, 0].float().numpy(), v[:, 0].float().numpy()
    want = [R.attention(q[:, h].double().numpy(), R.held(kf, group), R.held(vf, group),
                        R.step(kf, group), R.step(vf, group), np.array([n - 1]), 0.1, 0)
            for h in range(4)]
    R.check(out, lse, want, F16)


def test_decode_nan_query_stays_in_its_head(dkv_gpu):
    cache, table, end, _, _ = fill(dkv_gpu, [100], 1, 128, 32, 64, F16, 4)
    q = torch.randn(1, 8, 128, device="cuda", dtype=F16)
    ref = cache.decode_attn(q, 0.1, table, end)
    q[0, 3, 5] = float("nan")
    got = cache.decode_attn(q, 0.1, table, end)
    assert bool(torch.isnan(got[0, 3]).all())
    keep = [h for h in range(8) if h != 3]
    assert torch.equal(got[0, keep], ref[0, keep])


def test_stale_pages_are_not_seen(dkv_gpu):
    """Positions behind a sequence's length hold another sequence's leftovers."""
    cache, table, end, ks, vs = fill(dkv_gpu, [64], 1, 128, 32, 64, F16, 4)
    q = torch.randn(1, 4, 128, device="cuda", dtype=F16)
    for n in (1, 17, 40):
        short = torch.tensor([n], dtype=torch.int32, device="cuda")
        out = cache.decode_attn(q, 0.1, table, short)
        want = [R.attention(q[:, h].double().cpu().numpy(), R.held(ks[0][:n, 0], 32),
                            R.held(vs[0][:n, 0], 32), R.step(ks[0][:n, 0], 32),
                            R.step(vs[0][:n, 0], 32), np.array([n - 1]), 0.1, 0) for h in range(4)]
        R.check(out, None, want, F16)


def test_shared_prefix_pages(dkv_gpu):
    """Two sequences read the same pages."""
    cache, table, end, _, _ = fill(dkv_gpu, [64, 10], 2, 128, 32, 64, F16, 4)
    q = torch.randn(1, 8, 128, device="cuda", dtype=F16).expand(3, 8, 128)
    both = table[:1].expand(3, -1).contiguous()
    ends = torch.tensor([64, 50, 64], dtype=torch.int32, device="cuda")
    out = cache.decode_attn(q, 0.1, both, ends)
    one = cache.decode_attn(q[:1], 0.1, table[:1].contiguous(), ends[:1].clone())
    # (the work split differs with the batch, so the sums' order may)
    assert torch.equal(out[0], out[2]) or torch.allclose(out[0].float(), out[2].float(), rtol=2 ** -10, atol=2e-4)
    assert torch.allclose(out[0].float(), one[0].float(), rtol=2 ** -10, atol=2e-4)


def test_device_faults_set_the_status_word(dkv_gpu):
    cache, table, end, _, _ = fill(dkv_gpu, [100, 40], 2, 64, 32, 16, F16, 4)
    d = dkv_gpu
    q = torch.randn(2, 4, 64, device="cuda", dtype=F16)
    good = cache.decode_attn(q, 0.1, table, end)
    bad = table.clone()
    bad[0, 2] = 10 ** 6
    bad[0, 3] = -1
    out = cache.decode_attn(q, 0.1, bad, end)
    assert cache.device_status() == d.DEV_BAD_PAGE and cache.device_status() == 0
    assert bool(torch.isfinite(out).all())
    assert torch.allclose(out[1].float(), good[1].float(), rtol=2 ** -10, atol=2e-4)
    for n in (-1, 10 ** 6):
        ends = end.clone()
        ends[1] = n
        out = cache.decode_attn(q, 0.1, table, ends)
        assert cache.device_status() == d.DEV_BAD_SEQLEN
        assert not bool(out[1].any())
    k = torch.randn(6, 2, 64, device="cuda", dtype=F16)
    before = cache.pool.clone()
    for starts in ([0, 3, 2], [0, -4, 6], [4, 2, 6]):      # decreasing
        cache.append(k, k, table, end, torch.tensor(starts, dtype=torch.int32, device="cuda"))
        assert cache.device_status() == d.DEV_BAD_SEQLEN, starts
    short = torch.tensor([2, 40], dtype=torch.int32, device="cuda")   # 3 rows, 2 positions
    cache.pool.copy_(before)
    cache.append(k, k, table, short, torch.tensor([0, 3, 3], dtype=torch.int32, device="cuda"))
    assert cache.device_status() == d.DEV_BAD_SEQLEN
    assert torch.equal(cache.pool, before)
    cache.append(k[:2], k[:2], bad, torch.tensor([33, 0], dtype=torch.int32, device="cuda"),
                 torch.tensor([0, 2, 2], dtype=torch.int32, device="cuda"))
    assert cache.device_status() == d.DEV_BAD_PAGE


def test_starts_beyond_the_rows_given(dkv_gpu):
    """starts[batch] past n_rows: rows that do not exist are not touched."""
    cache, table, end, _, _ = fill(dkv_gpu, [20, 20], 1, 64, 32, 16, F16, 4)
    k = torch.randn(8, 1, 64, device="cuda", dtype=F16)
    cache.append(k[:5], k[:5], table, end, torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda"))
    a, b = cache.read(5, table, end, torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda"))
    assert np.array_equal(a.double().cpu().numpy(), R.held(k[:5].float().cpu().numpy(), 32))
    assert cache.device_status() == 0


def test_serving_steps_on_a_side_stream_and_in_a_graph(dkv_gpu):
    """Append and decode as a captured step, replayed as the lengths grow, and
    the same steps eagerly on another stream: equal bits."""
    H, G, D, page, B = 2, 4, 128, 16, 3
    lens = [5, 0, 30]
    steps = 20
    t = R.Tables([n + steps for n in lens], page, 6)
    table, _ = t.dev()
    rng = np.random.default_rng(1)
    ctx = [R.make_kv(rng, sum(lens), H, D, BF16).cuda() for _ in range(2)]
    news = torch.from_numpy(rng.normal(size=(steps, B, (G + 2) * H, D))).to(BF16).cuda()

    def fresh():
        c = dkv_gpu.Kv4Cache(t.n_pages, H, head_dim=D, page_size=page)
        end = torch.tensor(lens, dtype=torch.int32, device="cuda")
        c.append(*ctx, table, end, R.starts_of(lens))
        return c, end

    def one(c, x, end, stream=None):
        c.append(x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:], table, end, stream=stream)
        return c.decode_attn(x[:, :G * H], 0.09, table, end, stream=stream)

    c, end = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    eager = []
    with torch.cuda.stream(side):
        for i in range(steps):
            end += 1
            eager.append(one(c, news[i], end))
    torch.cuda.current_stream().wait_stream(side)

    c2, end2 = fresh()
    x = torch.empty_like(news[0])
    graph = torch.cuda.CUDAGraph()
    one(c2, news[0], end2 + 1)                 # (warm-up; position n is written again)
    with torch.cuda.graph(graph):
        end2 += 1
        y = one(c2, x, end2)
    for i in range(steps):
        x.copy_(news[i])
        graph.replay()
        assert torch.equal(y, eager[i]), i
    # a stream handed over, from another current stream
    c3, end3 = fresh()
    for i in range(2):
        end3 += 1
        side.wait_stream(torch.cuda.current_stream())
        z = one(c3, news[i], end3, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(z, eager[i])
    assert c.device_status() == c2.device_status() == c3.device_status() == 0
