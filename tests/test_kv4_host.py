"""CPU checks of the paged 4-bit cache: page sizes, the refusals of its C
functions before they touch the GPU, and the arithmetic that cuts a prompt
call's work into runs."""
import ctypes
import math
import random

import pytest

TM, TN, COST, MIN_TILES = 128, 128, 3, 6


@pytest.fixture(scope="module")
def dkv():
    from delta_quantized_kv_b200 import build
    build.build()
    import delta_quantized_kv_b200 as m
    m.load()
    return m


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [32, 64])
def test_page_bytes(dkv, D, group):
    for H, page in ((1, 16), (8, 64), (5, 48), (4096, 65536)):
        d = dkv.dkv_kv4_desc(H, D, group, page)
        assert dkv.dkv_kv4_page_bytes(d) == H * page * 2 * (D // 2 + 2 * D // group)


@pytest.mark.parametrize("bad", [(0, 128, 32, 64), (4097, 128, 32, 64), (8, 96, 32, 64), (8, 256, 32, 64),
                                 (8, 128, 16, 64), (8, 128, 128, 64), (8, 128, 32, 0), (8, 128, 32, 24),
                                 (8, 128, 32, 65552), (8, 128, 32, -16)])
def test_bad_descriptors(dkv, bad):
    d = dkv.dkv_kv4_desc(*bad)
    assert dkv.dkv_kv4_page_bytes(d) == 0
    with pytest.raises(dkv.DkvError):
        dkv.dkv_kv4_init(d, 4096, 4, 4096, 0)
    for nb in (dkv.dkv_kv4_decode_workspace_bytes(d, 1, 1, 8, 1),
               dkv.dkv_kv4_prompt_workspace_bytes(d, 1, 1, 8, 1, True)):
        assert nb == 0


# addresses that are never followed: every call below is refused
P = 1 << 20


def _pool(dkv, **kw):
    d = dkv.dkv_kv4_desc(2, 128, 32, 64)
    f = dict(base=P, n_pages=4, page_bytes=dkv.dkv_kv4_page_bytes(d), status=P)
    f.update(kw)
    return dkv.dkv_kv4_pool(d, f["base"], f["n_pages"], f["page_bytes"], f["status"])


def _seqs(dkv, **kw):
    f = dict(batch=2, max_pages=3, block_table=P, seq_lens=P, starts=P)
    f.update(kw)
    return dkv.dkv_kv4_batch(f["batch"], f["max_pages"], f["block_table"], f["seq_lens"], f["starts"])


def _calls(dkv, pool=None, seqs=None, n=4, nq=1, dtype=None, rows=P, stride=256, head=128, out=P, ws=P,
           nb=1 << 60, scale=0.1, window=0, Hq=4, lse=None):
    lib, b = dkv.load(), ctypes.byref
    pool, seqs = pool or _pool(dkv), seqs or _seqs(dkv)
    f16 = dkv.DKV_F16 if dtype is None else dtype
    return {
        "append": lambda: lib.dkv_kv4_append(b(pool), b(seqs), rows, P, f16, n, stride, head, 256, 128, 0),
        "append_v": lambda: lib.dkv_kv4_append(b(pool), b(seqs), P, rows, f16, n, 256, 128, stride, head, 0),
        "read": lambda: lib.dkv_kv4_read(b(pool), b(seqs), out, P, f16, n, 0),
        "decode": lambda: lib.dkv_kv4_decode_attn(b(pool), b(seqs), rows, f16, Hq, nq, stride, head, scale,
                                                  window, out, lse, ws, nb, 0),
        "prompt": lambda: lib.dkv_kv4_prompt_attn(b(pool), b(seqs), rows, f16, Hq, n, stride, head, scale,
                                                  window, out, lse, ws, nb, 0),
    }


ALL = ("append", "append_v", "read", "decode", "prompt")
ATTN = ("decode", "prompt")
ROWS = ("append", "append_v", "decode", "prompt")


def test_refused_pools_and_batches(dkv):
    E, A, C = dkv.DKV_EINVAL, dkv.DKV_EALIGN, dkv.DKV_ECAPACITY
    for kw, want in (({"base": None}, E), ({"status": None}, E), ({"n_pages": 0}, E), ({"n_pages": 1 << 31}, E),
                     ({"page_bytes": 1}, E), ({"base": P + 16}, A), ({"status": P + 2}, A)):
        calls = _calls(dkv, pool=_pool(dkv, **kw))
        for f in ALL:
            assert calls[f]() == want, (kw, f)
    for kw, want in (({"batch": 0}, E), ({"batch": 16385}, E), ({"max_pages": 0}, E), ({"block_table": None}, E),
                     ({"seq_lens": None}, E), ({"max_pages": 1 << 25}, C), ({"block_table": P + 2}, A),
                     ({"seq_lens": P + 1}, A)):
        calls = _calls(dkv, seqs=_seqs(dkv, **kw))
        for f in ALL:
            assert calls[f]() == want, (kw, f)
    calls = _calls(dkv, seqs=_seqs(dkv, starts=P + 2))
    for f in ("append", "read", "prompt"):
        assert calls[f]() == A
    # without starts the rows are shared out evenly
    calls = _calls(dkv, seqs=_seqs(dkv, starts=None), n=3)
    for f in ("append", "read", "prompt"):
        assert calls[f]() == E
    calls = _calls(dkv, n=0)
    for f in ("append", "read", "prompt"):
        assert calls[f]() == E


def test_refused_rows(dkv):
    E, A = dkv.DKV_EINVAL, dkv.DKV_EALIGN
    for kw, want in (({"rows": None}, E), ({"rows": P + 8}, A), ({"stride": 4}, A), ({"head": 129}, A),
                     ({"stride": -256}, E), ({"head": -128}, E), ({"dtype": 7}, E), ({"dtype": -1}, E)):
        calls = _calls(dkv, **kw)
        for f in ROWS:
            assert calls[f]() == want, (kw, f)
    for f in ("read", "decode", "prompt"):
        assert _calls(dkv, out=None)[f]() == E
        assert _calls(dkv, out=P + 4)[f]() == A


def test_refused_attention(dkv):
    E, A, C = dkv.DKV_EINVAL, dkv.DKV_EALIGN, dkv.DKV_ECAPACITY
    for kw, want in (({"Hq": 3}, E), ({"Hq": 0}, E), ({"scale": 0.0}, E), ({"scale": -1.0}, E),
                     ({"scale": math.inf}, E), ({"scale": math.nan}, E), ({"window": -1}, E), ({"ws": None}, E),
                     ({"ws": P + 8}, A), ({"lse": P + 2}, A), ({"dtype": dkv.DKV_F32}, dkv.DKV_EUNSUPPORTED)):
        calls = _calls(dkv, **kw)
        for f in ATTN:
            assert calls[f]() == want, (kw, f)
    for nq in (0, 17, -1):
        assert _calls(dkv, nq=nq)["decode"]() == E
    # more query rows, or runs of the decode step, than the grids take
    assert _calls(dkv, n=1 << 29, Hq=4)["prompt"]() == C
    assert _calls(dkv, seqs=_seqs(dkv, batch=16384), nq=16, Hq=2048)["decode"]() == C


# ---------------------------------------------------------------------------
# runs of a prompt call (the closed formulas of the kernel, in Python)
# ---------------------------------------------------------------------------
class Prompt:
    def __init__(self, seqs, H, G, window, ctas):
        self.H, self.G, self.w, self.seqs = H, G, window, seqs          # seqs: (len, n)
        self.cost = COST * TN * G
        self.jobs = []                                                  # (units, tiles)
        for b, (length, n) in enumerate(seqs):
            for _ in range(H):
                for i in range(self.blocks(n)):
                    self.jobs.append((self.at(b, i), self.tiles(b, i)))
        self.total = sum(u for u, _ in self.jobs)
        least = MIN_TILES * TN * G
        k = self.total // least
        self.n = int(self.total > 0) if k < 1 else min(k, ctas)

    def blocks(self, n):
        return -(-n * self.G // (2 * TM))

    def tiles(self, b, i):
        length, n = self.seqs[b]
        row0, nrow, pos0 = i * 2 * TM, n * self.G, length - n
        first, last = pos0 + row0 // self.G, pos0 + (min(row0 + 2 * TM, nrow) - 1) // self.G
        lo = max(0, first - self.w + 1) & ~15 if self.w else 0
        return -(-(last + 1 - lo) // TN)

    def base_full(self, b):
        length, n = self.seqs[b]
        return self.G * (length - n), self.G * self.w + 2 * TM if self.w else 2 ** 63 - 1

    def at(self, b, i):
        base, full = self.base_full(b)
        return min(full, base + 2 * TM * (i + 1)) + self.cost

    def before(self, b, m):
        base, full = self.base_full(b)
        k = 0 if full <= base else min(m, (full - base) // (2 * TM))
        return base * k + TM * k * (k + 1) + (m - k) * full * (m > k) + m * self.cost

    def unit_of(self, c):
        q, r = divmod(self.total, self.n)
        return c * q + min(c, r)

    def cta_of(self, u):
        q, r = divmod(self.total, self.n)
        return u // (q + 1) if u < r * (q + 1) else r + (u - r * (q + 1)) // q


def _upto(x, units, cost, tiles):
    each = (units - cost + tiles - 1) // tiles
    return 0 if x <= cost else tiles if x >= units else min(tiles, (x - cost) // each)


@pytest.mark.parametrize("seed", range(60))
def test_runs_of_a_prompt_call_cover_every_tile_once(seed):
    rng = random.Random(seed)
    G, H, window = rng.choice([1, 2, 3, 4, 7, 8, 64]), rng.choice([1, 2, 5]), rng.choice([0, 0, 1, 100, 3001])
    seqs = []
    for _ in range(rng.choice([1, 2, 9])):
        n = rng.choice([1, 2, 40, 255, 256, 700, 2500])
        seqs.append((n + rng.choice([0, 1, 500, 20000]), n))
    p = Prompt(seqs, H, G, window, rng.choice([1, 2, 148]))
    for b, (_, n) in enumerate(seqs):          # the closed sum is the sum
        for m in (0, 1, p.blocks(n) // 2, p.blocks(n)):
            assert p.before(b, m) == sum(p.at(b, i) for i in range(m))
    start = 0
    for units, tiles in p.jobs:
        end, at, shares = start + units, 0, []
        for c in range(p.cta_of(start), p.cta_of(end - 1) + 1):
            u0, u1 = max(p.unit_of(c), start) - start, min(p.unit_of(c + 1), end) - start
            t0, t1 = _upto(u0, units, p.cost, tiles), _upto(u1, units, p.cost, tiles)
            assert t0 == at and t1 >= t0
            at = t1
            if t1 > t0:
                shares.append(c)
        assert at == tiles
        # those that share a job follow one another up to the CTA of its last unit
        assert shares == list(range(shares[0], p.cta_of(end - 1) + 1))
        start = end
