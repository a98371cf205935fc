"""The paged 4-bit cache in numpy and 64 bits, for the tests: the block rule,
page tables, and attention over the held values."""
import math

import numpy as np
import torch


def quantise(x, group):
    """x: float32 [..., D] -> codes, zero points and scales ([..., D / group,
    group], [..., D / group]), by the block rule in numpy."""
    x = np.nan_to_num(np.asarray(x, np.float32), nan=0.0, posinf=np.inf, neginf=-np.inf)
    x = np.clip(x, np.float32(-32768), np.float32(32768)).reshape(
        *x.shape[:-1], x.shape[-1] // group, group)
    hi = np.maximum(x.max(-1), np.float32(0))
    lo = np.minimum(x.min(-1), np.float32(0))
    r = ((hi - lo) * (np.float32(1) / np.float32(15))).astype(np.float32)
    m, e = np.frexp(r.astype(np.float64))
    e = np.maximum(e - 7, -20)
    s = np.ldexp(np.ceil(np.ldexp(r.astype(np.float64), -e)), e)
    d = np.where(s > 0, s, 1.0).astype(np.float32)
    zero = np.minimum(15, np.rint((-lo / d).astype(np.float32)))
    code = np.clip(np.rint((x / d[..., None]).astype(np.float32)) + zero[..., None], 0, 15)
    none = s == 0
    zero[none] = 0
    code[none] = 0
    return code, zero, s


def held(x, group):
    """The values held for x [..., D], float64."""
    code, zero, s = quantise(x, group)
    return ((code - zero[..., None]) * s[..., None]).reshape(*np.shape(x))


def step(x, group):
    """15 s of each channel's block: bounds code s and zero s."""
    s = quantise(x, group)[2]
    return np.repeat(15.0 * s, group, axis=-1)


class Tables:
    """A shuffled block table for sequences of the given lengths."""

    def __init__(self, lens, page, seed=0, spare=2, width=None):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + spare
        perm = rng.permutation(self.n_pages)
        width = max(1, max(need)) if width is None else width
        # entries that no position needs are out of range on purpose
        self.table = np.full((len(lens), width), -7, np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = perm[at:at + k]
            at += k
        self.lens = np.asarray(lens, np.int32)

    def dev(self):
        return torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda()


def starts_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()


def make_kv(rng, rows, heads, dim, dtype):
    spread = np.exp(rng.uniform(math.log(0.2), math.log(3.0), (heads, dim)))
    far = (rng.random((heads, dim)) < 0.1) * rng.normal(size=(heads, dim)) * 4
    x = torch.from_numpy((rng.normal(size=(rows, heads, dim)) * spread + far).astype(np.float32))
    return x.to(dtype)


def attention(q, k, v, k15, v15, pos, scale, window):
    """One kv head in float64: q [n, D] at positions pos [n]; k, v [L, D] the
    held values, k15, v15 = step() of them.  Returns out, lse, and the bounds
    below of a 16-bit kernel's errors before its own output rounding, by
    (weights rounded to fp16 once; weights times scales rounded again) and of
    lse."""
    L = k.shape[0]
    at = np.arange(L)[None]
    seen = at <= pos[:, None]
    if window:
        seen &= at > pos[:, None] - window
    x = np.where(seen, scale * (q @ k.T), -np.inf)
    top = x.max(-1, keepdims=True) if L else np.full((len(q), 1), -np.inf)
    top = np.where(np.isinf(top), 0.0, top)
    w = np.exp(x - top)
    tot = w.sum(-1, keepdims=True)
    div = np.where(tot > 0, tot, 1.0)
    p = w / div
    with np.errstate(divide="ignore"):
        lse = (np.log(tot) + top)[:, 0]
    # scores: sums of up to 2 x 128 products in fp32 whose terms are code s q and
    # zero s q, each at most 15 s |q|; 2^-20 covers 2^-24 a term in any order of
    # 16 partial sums, and ex2's own 2^-22
    eps = 2.0 ** -20 * (1 + scale * (np.abs(q) @ k15.T))
    eps = np.where(seen, eps, 0.0).max(-1, keepdims=True) if L else np.zeros((len(q), 1))
    a, b = p @ np.abs(v), p @ v15
    # the tensor core truncates: an MMA's 16 products and its accumulator are
    # aligned to the largest and cut to 24 bits, so each of the 17 loses at most
    # 2^-23 of it.  The products of all MMAs together: <= 17 * 2^-23 * b, as no
    # product passes the sum b of all; the accumulator, once in each of the two
    # MMAs (hi and lo) of every 16 positions: <= 2^-23 * b.  Twice: codes and
    # zero points are summed apart
    mmas = 2 * -(-L // 16)
    once = 2.0 ** -11 * a + 2 * eps * a + 2 * (17 * 2 + mmas) * 2.0 ** -23 * b
    twice = once + 2.0 ** -11 * b
    return p @ v, lse, once, twice, eps[:, 0] + 2.0 ** -21 * (1 + np.abs(np.where(tot > 0, lse[:, None], 0)))[:, 0]


def check(out, lse, want, dtype, exact_values=False):
    """out [n, heads, D] and lse [n, heads] of a kernel against want, a list per
    head of attention()'s results.  exact_values: the kernel multiplies the
    weights with the held values themselves, in either type."""
    u = torch.finfo(dtype).eps / 2
    out = out.float().cpu().numpy().astype(np.float64)
    for h, (o, l, once, twice, le) in enumerate(want):
        # half a step of the output type, and fp16's subnormals below it
        tol = (twice if dtype == torch.bfloat16 and not exact_values else once) * (1 + u) + u * np.abs(o) + 2.0 ** -25
        bad = ~(np.abs(out[:, h] - o) <= tol)
        assert not bad.any(), (h, np.argwhere(bad)[:4], out[:, h][bad][:4], o[bad][:4], tol[bad][:4])
        if lse is not None:
            x = lse[:, h].cpu().numpy().astype(np.float64)
            assert np.array_equal(np.isneginf(x), np.isneginf(l))
            f = ~np.isneginf(l)
            assert np.all(np.abs(x[f] - l[f]) <= le[f]), (h, np.abs(x[f] - l[f]).max(), le[f].min())
