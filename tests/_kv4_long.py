"""Long sequences of the paged 4-bit cache, for the tests: values that mark the
place they stand at, and bounds that grow with the positions one accumulator
runs through instead of the whole length."""
import math

import numpy as np
import torch

import _kv4 as R


def marked_kv(rng, rows, heads, dim, dtype):
    """Keys as in make_kv; values that are 1 in one channel, another every rows /
    dim positions, and 0 elsewhere: a channel of the output is the weight of its
    stretch of positions.  (Their zero points are 0.)"""
    k = R.make_kv(rng, rows, heads, dim, dtype)
    v = np.zeros((rows, heads, dim), np.float32)
    at = np.arange(rows) // max(1, -(-rows // dim))
    for h in range(heads):
        v[np.arange(rows), h, (at + 7 * h) % dim] = 1.0
    return k, torch.from_numpy(v).to(dtype)


def terms(v, v15, exact_values):
    """What a weight is multiplied with, for v15 in the bounds: the value held, or
    code * scale.  Of marked values that is the value held too (zero point 0), but
    at odd positions, which are stored mirrored: code 15 - c, zero point 15, scale
    -s.  There both products are at most 15 s."""
    odd = np.arange(len(v))[:, None] % 2 == 1
    return v if exact_values else np.where(odd, v15, v)


def decode_chain(lens, H, G, nq, sms):
    """(positions of a warp's run, records that are joined for an output)."""
    units = sum(-(-n // 32) for n in lens) * H * -(-nq * G // 8)
    warps = max(1, min(-(-units // 2), 16 * sms))
    run = -(-units // warps)
    return 32 * run, 8 + -(-max(lens) // 32) // max(1, 8 * (units // warps)) + 3


def prompt_chain(seqs, H, G, sms):
    """The same of a prompt call of (length, rows) without a window; (several tiles
    of 128 positions a CTA)."""
    total = 0
    for length, n in seqs:
        blocks = -(-n * G // 256)
        total += H * sum(G * (length - n) + 256 * (i + 1) + 3 * 128 * G for i in range(blocks))
    ctas = max(1, min(total // (6 * 128 * G), sms))
    tiles = -(-total // ctas) // (128 * G) + 2
    return 128 * tiles, -(-max(length for length, _ in seqs) // (128 * max(1, tiles - 4))) + 3


def attention(q, k, v, k15, v15, pos, scale, window, chain, joins):
    """attention() of _kv4 with its bounds taken for accumulators that run through
    `chain` positions each, `joins` of them added up in fp32."""
    at = np.arange(k.shape[0])[None]
    seen = at <= pos[:, None]
    if window:
        seen &= at > pos[:, None] - window
    x = np.where(seen, scale * (q @ k.T), -np.inf)
    top = x.max(-1, keepdims=True)
    w = np.exp(x - top)
    tot = w.sum(-1, keepdims=True)
    p = w / tot
    lse = (np.log(tot) + top)[:, 0]
    eps = 2.0 ** -20 * (1 + scale * (np.abs(q) @ k15.T))
    eps = np.where(seen, eps, 0.0).max(-1, keepdims=True)
    a, b = p @ np.abs(v), p @ v15
    mmas = 2 * -(-chain // 16)
    # joining: two products and a sum of each part, 2^-24 of what has been added up
    once = 2.0 ** -11 * a + 2 * eps * a + (2 * (17 * 2 + mmas) + 3 * joins / 2) * 2.0 ** -23 * b
    twice = once + 2.0 ** -11 * b
    return p @ v, lse, once, twice, eps[:, 0] + 2.0 ** -21 * (1 + np.abs(lse))


def tight(want, dtype, exact_values):
    """The largest tolerance check() allows, as a part of the mean output."""
    u = torch.finfo(dtype).eps / 2
    r = 0.0
    for o, _, once, twice, _ in want:
        tol = (twice if dtype == torch.bfloat16 and not exact_values else once) * (1 + u) + u * np.abs(o) + 2.0 ** -25
        r = max(r, float(tol.max() / np.abs(o).mean()))
    return r


def half_a_share(rows, dim):
    """Half of what the least share of a warp (64 positions) has of a channel's output."""
    return 32 / -(-rows // dim)


def softmax_scale(dim):
    return 0.5 / math.sqrt(dim)
