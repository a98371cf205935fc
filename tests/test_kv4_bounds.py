"""CPU check of the long tests' bounds: an output that misses the positions of
one run, or counts them twice, is out of them."""
import numpy as np
import pytest
import torch

import _kv4 as R
import _kv4_long as long


@pytest.mark.parametrize("kind,D,group,dtype", [("decode", 128, 32, torch.float16), ("decode", 64, 64, torch.bfloat16),
                                                ("prompt", 128, 64, torch.bfloat16), ("prompt", 64, 32, torch.float16)])
def test_a_lost_or_doubled_run_is_out_of_bounds(kind, D, group, dtype):
    rng = np.random.default_rng(D + group)
    L, H, G = 70001, 1, 4
    k, v = (x.float().numpy()[:, 0] for x in long.marked_kv(rng, L, H, D, dtype))
    chain, joins = long.decode_chain([L, 9000], 2, 8, 1, 148) if kind == "decode" else \
        long.prompt_chain([(L, 3), (9000, 1)], 2, 8, 148)
    assert chain < 2500 and joins < 200
    scale, q = long.softmax_scale(D), rng.normal(size=(G, D))
    pos = np.full(G, L - 1)
    hk, hv = R.held(k, group), R.held(v, group)
    exact = kind == "prompt"
    v15 = long.terms(hv, R.step(v, group), exact)
    want = [long.attention(q[h:h + 1], hk, hv, R.step(k, group), v15, pos[h:h + 1], scale, 0, chain, joins)
            for h in range(G)]
    assert long.tight(want, dtype, exact) < long.half_a_share(L, D)

    def outs(f, g):           # weights times f above, times g below
        y = np.empty((1, G, D))
        for h in range(G):
            w = np.exp(scale * (hk @ q[h]) - want[h][1][0])
            y[0, h] = (w * f) @ hv / (w * g).sum()
        return torch.from_numpy(y).to(dtype)

    one = np.ones(L)
    R.check(outs(one, one), None, want, dtype, exact_values=exact)
    for length in (chain, 64):                # a run; the least a warp takes
        for start in rng.integers(0, L - length, 6) // 32 * 32:
            for factor in (0.0, 2.0):
                f = one.copy()
                f[start:start + length] = factor
                for g in (one, f):
                    with pytest.raises(AssertionError):
                        R.check(outs(f, g), None, want, dtype, exact_values=exact)
