"""Decode and prompt attention over long sequences of the paged 4-bit cache,
whose work many warps and CTAs share: values that mark their place show a lost
or doubled share (test_kv4_bounds.py)."""
import numpy as np
import pytest
import torch

import _kv4 as R
import _kv4_long as long
from test_gpu_kv4 import BF16, F16

pytestmark = pytest.mark.gpu


def filled(dkv, lens, H, D, group, page, dtype, seed):
    rng = np.random.default_rng(seed)
    t = R.Tables(lens, page, seed)
    cache = dkv.Kv4Cache(t.n_pages, H, head_dim=D, page_size=page, group=group)
    table, end = t.dev()
    kv = [long.marked_kv(rng, n, H, D, dtype) for n in lens]
    cache.append(*(torch.cat([x[i] for x in kv]).cuda() for i in range(2)), table, end, R.starts_of(lens))
    held = [tuple(R.held(x.float().numpy(), group) for x in pair) for pair in kv]
    steps = [tuple(R.step(x.float().numpy(), group) for x in pair) for pair in kv]
    return cache, table, end, held, steps, rng


def check(out, lse, q, held, steps, lens, scale, window, chain, joins, dtype, exact):
    """out, q [sequence][row]: the rows' positions are the last of each sequence."""
    for b, n in enumerate(lens):
        m = q[b].shape[0]
        qf = q[b].double().cpu().numpy()
        want = []
        for h in range(q[b].shape[1]):
            kvh = h // (q[b].shape[1] // held[b][0].shape[1])
            (k, v), (k15, v15) = ((x[:, kvh] for x in pair) for pair in (held[b], steps[b]))
            want.append(long.attention(qf[:, h], k, v, k15, long.terms(v, v15, exact), n - m + np.arange(m),
                                       scale, window, chain, joins))
        assert n < 60000 or window or long.tight(want, dtype, exact) < long.half_a_share(n, out[b].shape[-1])
        R.check(out[b], lse[b], want, dtype, exact_values=exact)


@pytest.mark.parametrize("D,group,dtype", [(128, 32, F16), (128, 64, BF16), (64, 32, BF16), (64, 64, F16)])
@pytest.mark.parametrize("nq,window", [(1, 0), (1, 50001), (3, 0)])
def test_decode(dkv_gpu, D, group, dtype, nq, window):
    lens, H, G = [70001, 9000, 333], 2, 8
    cache, table, end, held, steps, rng = filled(dkv_gpu, lens, H, D, group, 64, dtype, D + nq)
    q = torch.from_numpy(rng.normal(size=(len(lens), nq, H * G, D))).to(dtype).cuda()
    scale = long.softmax_scale(D)
    out, lse = cache.decode_attn(q, scale, table, end, window=window, return_lse=True)
    assert cache.device_status() == 0
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    chain, joins = long.decode_chain(lens, H, G, nq, sms)
    check(out, lse, q, held, steps, lens, scale, window, chain, joins, dtype, False)


@pytest.mark.parametrize("D,group,dtype", [(128, 32, F16), (128, 64, BF16), (64, 32, BF16), (64, 64, F16)])
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 3, 17]])
def test_prompt(dkv_gpu, D, group, dtype, new):
    lens, H, G = [70001, 9000, 333], 2, 8
    cache, table, end, held, steps, rng = filled(dkv_gpu, lens, H, D, group, 64, dtype, D + new[0])
    q = torch.from_numpy(rng.normal(size=(sum(new), H * G, D))).to(dtype).cuda()
    scale = long.softmax_scale(D)
    out, lse = cache.prompt_attn(q, scale, table, end, R.starts_of(new), return_lse=True)
    assert cache.device_status() == 0
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    chain, joins = long.prompt_chain(list(zip(lens, new)), H, G, sms)
    out, lse, q = (torch.split(x, new) for x in (out, lse, q))
    check(out, lse, q, held, steps, lens, scale, 0, chain, joins, dtype, True)
