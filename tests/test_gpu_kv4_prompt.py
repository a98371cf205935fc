"""Prompt attention over the paged 4-bit cache against float64: ragged chunks
behind contexts of any length, windows, odd head groups, few rows over long
contexts (split positions), padding, faults, and a run of the operators as a
server uses them."""
import math

import numpy as np
import pytest
import torch

import _kv4 as R
from test_gpu_kv4 import BF16, F16, F32, fill

pytestmark = pytest.mark.gpu


def prompt_case(dkv, lens, new, H, G, D, group, page, dtype, window=0, seed=0, gain=1.0, pad=0,
                every=1, scale=None, width=None):
    """lens: positions held; new: the last of them that ask.  Checks every
    `every`-th row (and the last)."""
    cache, table, end, ks, vs = fill(dkv, lens, H, D, group, page, dtype, seed)
    if width:                      # a wide table, of which little is used
        table = torch.nn.functional.pad(table, (0, width - table.shape[1]), value=-1)
    rng = np.random.default_rng(seed + 1)
    scale = 1 / math.sqrt(D) if scale is None else scale
    n = sum(new)
    fused = torch.from_numpy(rng.normal(size=(n + pad, (G + 1) * H, D)) * gain).to(dtype).cuda()
    q = fused[:, :G * H]
    out = torch.full((n + pad, G * H, D), -5.0, dtype=dtype, device="cuda")
    out, lse = cache.prompt_attn(q, scale, table, end, R.starts_of(new), window=window, out=out,
                                 return_lse=True)
    assert cache.device_status() == 0
    assert bool((out[n:] == -5).all())
    qf, row = q.double().cpu().numpy(), 0
    for b, m in enumerate(new):
        at = sorted(set(range(0, m, every)) | ({m - 1} if m else set()))
        if at:
            want = []
            for h in range(G * H):
                k, v = ks[b][:, h // G], vs[b][:, h // G]
                want.append(R.attention(qf[[row + i for i in at], h], R.held(k, group),
                                        R.held(v, group), R.step(k, group), R.step(v, group),
                                        lens[b] - m + np.array(at), scale, window))
            R.check(out[row:row + m][at], lse[row:row + m][at], want, dtype, exact_values=True)
        row += m


@pytest.mark.parametrize("D,group", [(128, 32), (128, 64), (64, 32), (64, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_one_small_prompt(dkv_gpu, D, group, dtype):
    prompt_case(dkv_gpu, [100], [100], 1, 1, D, group, 64, dtype, seed=D)


@pytest.mark.parametrize("D,group", [(128, 32), (128, 64), (64, 32), (64, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("page,H,G", [(16, 1, 1), (64, 2, 4), (48, 3, 7)])
def test_ragged_chunks(dkv_gpu, D, group, dtype, page, H, G):
    lens = [1, 300, 0, 16, 129, 260, 40, 513, 128]
    new = [1, 7, 0, 16, 129, 200, 0, 100, 1]
    prompt_case(dkv_gpu, lens, new, H, G, D, group, page, dtype, seed=D + page, pad=3, every=3)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 100, 128, 129, 100000])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_window(dkv_gpu, window, dtype):
    prompt_case(dkv_gpu, [5, 400, 700], [5, 150, 33], 2, 3, 64, 32, 16, dtype, window, seed=window,
                every=2)


def test_whole_prompt_over_many_tiles(dkv_gpu):
    prompt_case(dkv_gpu, [2085], [2085], 2, 4, 128, 32, 64, BF16, seed=2, every=97)
    prompt_case(dkv_gpu, [1500, 900], [1500, 900], 1, 5, 128, 64, 32, F16, seed=3, every=61)


@pytest.mark.parametrize("new", [[1, 1], [3, 40], [200, 64]])
@pytest.mark.parametrize("window", [0, 3000])
def test_few_rows_over_long_contexts(dkv_gpu, new, window):
    """The positions are split over the grid and joined."""
    prompt_case(dkv_gpu, [9001, 4097], new, 2, 4, 128, 32, 64, F16, window, seed=4, every=37)


def test_short_contexts_in_a_wide_table(dkv_gpu):
    """Splits whose share of the positions is empty."""
    prompt_case(dkv_gpu, [3, 130, 0, 20], [2, 5, 0, 20], 1, 2, 128, 32, 16, F16, seed=5, width=4000)


def test_many_short_prompts(dkv_gpu):
    lens = [(11 * i) % 97 for i in range(80)]
    new = [n if i % 3 else n // 2 for i, n in enumerate(lens)]
    prompt_case(dkv_gpu, lens, new, 2, 2, 64, 64, 16, BF16, seed=6, every=5)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("gain", [1e-4, 30.0, 1000.0])
def test_query_magnitudes(dkv_gpu, dtype, gain):
    """From a flat softmax to rows whose maximum jumps by thousands."""
    prompt_case(dkv_gpu, [500], [300], 1, 4, 128, 32, 64, dtype, seed=7, gain=gain, every=7)


def test_uniform_rows_per_sequence(dkv_gpu):
    """starts=None: the same number of rows each."""
    lens, m, H, G, D = [50, 33], 9, 1, 4, 128
    cache, table, end, ks, vs = fill(dkv_gpu, lens, H, D, 32, 16, F16, 8)
    q = torch.randn(2 * m, G, D, device="cuda", dtype=F16)
    a = cache.prompt_attn(q, 0.1, table, end)
    b = cache.prompt_attn(q, 0.1, table, end, R.starts_of([m, m]))
    assert torch.equal(a, b)


def test_nan_query_stays_in_its_row(dkv_gpu):
    cache, table, end, _, _ = fill(dkv_gpu, [300], 1, 128, 32, 64, F16, 4)
    q = torch.randn(200, 4, 128, device="cuda", dtype=F16)
    ref = cache.prompt_attn(q, 0.1, table, end)
    q[77, 2, 5] = float("nan")
    got = cache.prompt_attn(q, 0.1, table, end)
    assert bool(torch.isnan(got[77, 2]).all())
    got[77, 2] = ref[77, 2]
    assert torch.equal(got, ref)


def test_device_faults_set_the_status_word(dkv_gpu):
    d = dkv_gpu
    lens, new, H, D = [200, 140], [60, 50], 1, 64
    cache, table, end, ks, vs = fill(d, lens, H, D, 32, 16, F16, 4)
    q = torch.randn(110, 2, D, device="cuda", dtype=F16)
    starts = R.starts_of(new)
    good = cache.prompt_attn(q, 0.1, table, end, starts)
    # a page that is not there: its 16 positions are not seen
    bad = table.clone()
    bad[0, 3] = 10 ** 6
    out, lse = cache.prompt_attn(q, 0.1, bad, end, starts, return_lse=True)
    assert cache.device_status() == d.DEV_BAD_PAGE
    assert torch.equal(out[60:], good[60:])
    keep = [i for i in range(200) if not 48 <= i < 64]
    k, v = R.held(ks[0][:, 0], 32), R.held(vs[0][:, 0], 32)
    x = 0.1 * q[59, 1].double().cpu().numpy() @ k[keep].T
    p = np.exp(x - x.max())
    # one fp16 rounding of each weight, one of the output (as in _kv4.attention)
    tol = 2.0 ** -10 * (p @ np.abs(v[keep]) / p.sum()) + 2.0 ** -10 * np.abs(p @ v[keep] / p.sum()) + 1e-5
    assert np.all(np.abs(out[59, 1].double().cpu().numpy() - p @ v[keep] / p.sum()) <= tol)
    # skipped sequences leave their rows alone
    for ends, st in (([200, -1], [0, 60, 110]), ([200, 10 ** 6], [0, 60, 110]),
                     ([200, 49], [0, 60, 110]), ([200, 140], [0, 60, 111]), ([200, 140], [0, 60, 5])):
        out = torch.full_like(good, -5)
        cache.prompt_attn(q, 0.1, table, torch.tensor(ends, dtype=torch.int32, device="cuda"),
                          torch.tensor(st, dtype=torch.int32, device="cuda"), out=out)
        assert cache.device_status() == d.DEV_BAD_SEQLEN, (ends, st)
        assert bool((out[60:] == -5).all())


def test_prompt_then_decode_agree(dkv_gpu):
    """A chunk of one row each is the decode step: the two kernels' answers
    differ by their roundings only."""
    lens, H, G, D = [77, 1, 300, 1025], 2, 4, 128
    cache, table, end, ks, vs = fill(dkv_gpu, lens, H, D, 32, 16, F16, 11)
    q = torch.randn(4, G * H, D, device="cuda", dtype=F16)
    a, la = cache.prompt_attn(q, 0.09, table, end, return_lse=True)
    b, lb = cache.decode_attn(q, 0.09, table, end, return_lse=True)
    for i, n in enumerate(lens):
        want = [R.attention(q[i:i + 1, h].double().cpu().numpy(), R.held(ks[i][:, h // G], 32),
                            R.held(vs[i][:, h // G], 32), R.step(ks[i][:, h // G], 32),
                            R.step(vs[i][:, h // G], 32), np.array([n - 1]), 0.09, 0)
                for h in range(G * H)]
        R.check(a[i:i + 1], la[i:i + 1], want, F16, exact_values=True)
        R.check(b[i:i + 1], lb[i:i + 1], want, F16)


def test_a_server_run(dkv_gpu):
    """Three requests: prompts in two ragged chunks, then decode steps, then a
    fourth that shares the first one's prefix pages; the last step captured into
    a graph.  Every output against float64 over the values read back."""
    H, G, D, page = 2, 4, 128, 16
    rng = np.random.default_rng(12)
    total = [150, 47, 90, 80]
    t = R.Tables(total, page, 12)
    t.table[3, :4] = t.table[0, :4]              # 64 positions shared
    table = torch.from_numpy(t.table).cuda()
    cache = dkv_gpu.Kv4Cache(t.n_pages, H, head_dim=D, page_size=page)
    x = [torch.from_numpy(rng.normal(size=(n, (G + 2) * H, D))).to(BF16).cuda() for n in total]
    x[3][:64] = x[0][:64]
    split = lambda y: (y[:, :G * H], y[:, G * H:(G + 1) * H], y[:, (G + 1) * H:])  # noqa: E731
    at = [0, 0, 0, 64]
    scale = 0.088
    outs = [[None] * n for n in total]

    def chunk(counts):
        y = torch.cat([x[b][at[b]:at[b] + c] for b, c in enumerate(counts)])
        for b, c in enumerate(counts):
            at[b] += c
        end = torch.tensor([a if c else 0 for a, c in zip(at, counts)], dtype=torch.int32).cuda()
        q, k, v = split(y)
        starts = R.starts_of(counts)
        cache.append(k, v, table, end, starts)
        o, row = cache.prompt_attn(q, scale, table, end, starts), 0
        for b, c in enumerate(counts):
            for i in range(c):
                outs[b][at[b] - c + i] = o[row + i]
            row += c

    chunk([100, 17, 0, 0])
    chunk([20, 20, 60, 10])
    stop = [total[0] - 1] + total[1:]            # request 0's last step is the captured one
    while any(a < n for a, n in zip(at, stop)):
        live = [b for b in range(4) if at[b] < stop[b]]
        y = torch.stack([x[b][at[b]] for b in live])
        for b in live:
            at[b] += 1
        end = torch.tensor([at[b] for b in live], dtype=torch.int32).cuda()
        q, k, v = split(y)
        tb = table[live].contiguous()
        cache.append(k, v, tb, end)
        o = cache.decode_attn(q, scale, tb, end)
        for i, b in enumerate(live):
            outs[b][at[b] - 1] = o[i]
    y = x[0][at[0]:at[0] + 1].clone()
    end = torch.tensor([total[0]], dtype=torch.int32).cuda()
    one = table[:1].contiguous()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, k, v = split(y)
        cache.append(k, v, one, end)
        o = cache.prompt_attn(q, scale, one, end)
    g.replay()
    outs[0][total[0] - 1] = o[0]
    assert cache.device_status() == 0
    for b in range(4):
        e = torch.tensor([total[b]], dtype=torch.int32).cuda()
        kk, vv = cache.read(total[b], table[b:b + 1].contiguous(), e, dtype=F32)
        raw = [z.float().cpu().numpy() for z in split(x[b])[1:]]
        for z, w in zip((kk, vv), raw):
            assert np.array_equal(z.cpu().numpy(), R.held(w, 32).astype(np.float32))
        rows = [i for i in range(total[b]) if outs[b][i] is not None]
        o = torch.stack([outs[b][i] for i in rows])
        q = split(x[b])[0].double().cpu().numpy()
        want = [R.attention(q[rows, h], R.held(raw[0][:, h // G], 32), R.held(raw[1][:, h // G], 32),
                            R.step(raw[0][:, h // G], 32), R.step(raw[1][:, h // G], 32),
                            np.array(rows), scale, 0) for h in range(G * H)]
        R.check(o, None, want, BF16)
