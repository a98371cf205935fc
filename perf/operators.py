"""The operators of the paged 4-bit cache, as measured: cases, inputs, a plain
form in elementary torch operations, and the definition in 64 bits.

  write   quantise new keys and values into the pages, and read them back
  read    read cached positions back as floating values
  decode  attention of one to a few new queries per sequence over the pages
  prompt  attention of ragged prompt chunks over the pages

A block is `group` channels of one token, kv head and tensor.  With x as fp32,
hi = max(0, max x) and lo = min(0, min x): r = (hi - lo) * (1/15) in fp32, s =
r rounded up to 7 significant bits (to a multiple of 2^-20 below 2^-14), zp =
min(15, rint(-lo / s)), code = clamp(rint(x / s) + zp, 0, 15), and the value
held is (code - zp) * s, which fp16 holds exactly.  s = 0 gives code = zp = 0.
"""
import math

import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def _case(name, op, dtype, batch, ctx, new, kv_heads, q_per_kv, head_dim, group, page, window=0, ragged=True,
          lse=False):
    """ctx: positions held before the call; new: tokens of the call (written, read or asked about); both per
    sequence, the largest of the batch where ragged."""
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "ctx": ctx, "new": new, "kv_heads": kv_heads,
            "q_per_kv": q_per_kv, "head_dim": head_dim, "group": group, "page": page, "window": window,
            "ragged": ragged, "lse": lse}


def listed():
    return [
        # one generated token of each of 64 running sequences: the smallest call, latency
        _case("write_tokens", "write", "bf16", 64, 4096, 1, 8, 4, 128, 32, 64, ragged=False),
        # a batch of prompts as they arrive
        _case("write_prompts", "write", "fp16", 4, 0, 8192, 8, 4, 128, 32, 64),
        # small heads, fp32 activations, pages of 48 tokens, odd chunk lengths behind odd contexts
        _case("write_chunks_d64", "write", "fp32", 7, 333, 1021, 4, 2, 64, 64, 48),
        # a shared prefix handed to another engine
        _case("read_prefix", "read", "bf16", 8, 0, 16384, 8, 4, 128, 32, 64, ragged=False),
        # odd ranges behind odd contexts, as fp32 for an error report
        _case("read_ranges_d64", "read", "fp32", 9, 517, 2049, 8, 2, 64, 32, 16),
        # one user, one token: latency
        _case("decode_single", "decode", "bf16", 1, 4095, 1, 8, 4, 128, 32, 64, ragged=False),
        # the decode step of a full batch at long context
        _case("decode_batch", "decode", "bf16", 16, 32767, 1, 8, 8, 128, 32, 64, ragged=False),
        # four draft tokens per sequence checked at once, ragged lengths, one of them empty, small pages
        _case("decode_draft", "decode", "fp16", 12, 16001, 4, 8, 4, 128, 64, 16, lse=True),
        # a sliding window over long ragged contexts, small heads
        _case("decode_window_d64", "decode", "fp16", 48, 30011, 1, 8, 7, 64, 32, 32, window=4096),
        # one long prompt from its beginning
        _case("prompt_whole", "prompt", "bf16", 1, 0, 8192, 8, 4, 128, 32, 64, ragged=False),
        # a chunk of a prompt behind a long prefix
        _case("prompt_chunk", "prompt", "fp16", 2, 24577, 500, 8, 4, 128, 64, 64),
        # many short prompts with a sliding window, an odd number of heads, small heads
        _case("prompt_short_d64", "prompt", "bf16", 24, 130, 777, 5, 3, 64, 32, 16, window=300, lse=True),
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["write", "read", "decode", "decode", "prompt", "prompt"])
    dtype = rng.choice(["fp16", "bf16"] if op in ("decode", "prompt") else ["fp16", "bf16", "fp32"])
    head_dim = rng.choice([64, 128, 128])
    group = rng.choice([32, 64])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    q_per_kv = rng.choice([1, 2, 3, 4, 6, 7, 8])
    window = 0
    if op in ("write", "read"):
        batch, new = size(1, 64), size(1, 16384)
        new = min(new, max(1, 280000 // (batch * kv_heads)))
        ctx = size(1, 4000) - 1
    elif op == "decode":
        batch, new = size(1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8])
        ctx = size(64, 60000)
        ctx = min(ctx, max(64, 500000 * 8 // (batch * kv_heads)))
        window = rng.choice([0, 0, 0, size(1, 8000)])
    else:
        batch, new = size(1, 32), size(1, 6000)
        new = min(new, int(math.sqrt(1.5e9 / (batch * kv_heads * q_per_kv))), 1_200_000 // (batch * kv_heads * q_per_kv))
        ctx = size(1, 24000) - 1
        ctx = min(ctx, max(0, 60_000_000 * 4 // (new * batch * kv_heads * q_per_kv) - new))
        window = rng.choice([0, 0, 0, size(1, 4000)])
    return {"op": op, "dtype": dtype, "batch": batch, "ctx": ctx, "new": new, "kv_heads": kv_heads,
            "q_per_kv": q_per_kv, "head_dim": head_dim, "group": group, "page": page, "window": window,
            "ragged": rng.random() < 0.7, "lse": rng.random() < 0.3}


def _sizes(case):
    """Per sequence: positions held with the call's tokens (end), and the call's tokens (new)."""
    end, new = [], []
    for i in range(case["batch"]):
        n, c = case["new"], case["ctx"]
        if case["ragged"]:
            f, g = (i * 0.6180339887) % 1.0, (i * 0.7548776662) % 1.0
            c = int(c * (1.0 - 0.75 * f))
            if case["op"] != "decode":
                n = max(1, int(n * (1.0 - 0.9 * g)))
            if i % 8 == 5:  # an empty sequence
                c, n = 0, n if case["op"] == "decode" else 0
        end.append(c + n if not (case["op"] == "decode" and case["ragged"] and i % 8 == 5) else 0)
        new.append(n)
    return end, new


def _visible(case):
    """Per sequence (query-position pairs, positions that some query sees)."""
    end, new = _sizes(case)
    w, pairs, span = case["window"], [], []
    for e, n in zip(end, new):
        n = min(n, e)
        first = e - n
        if w:
            k = max(0, min(n, w - first))   # queries that see less than the window
            pairs.append(k * first + k * (k + 1) // 2 + (n - k) * w)
            span.append(e - max(0, first - w + 1) if n else 0)
        else:
            pairs.append(n * first + n * (n + 1) // 2)
            span.append(e if n else 0)
    return pairs, span


def work(case):
    H, G, D = case["kv_heads"], case["q_per_kv"], case["head_dim"]
    size = 4 if case["dtype"] == "fp32" else 2
    row4 = H * 2 * (D // 2 + 2 * (D // case["group"]))   # packed bytes of one position
    row = H * 2 * D * size
    end, new = _sizes(case)
    n = sum(new)
    if case["op"] == "write":                            # in, packed, and back
        return {"bytes": n * (row + 2 * row4 + row), "flops": n * H * 2 * D * 6}
    if case["op"] == "read":
        return {"bytes": n * (row4 + row), "flops": n * H * 2 * D * 2}
    pairs, span = _visible(case)
    io = n * H * G * (2 * D * size + (4 if case["lse"] else 0))
    return {"bytes": sum(span) * row4 + io, "flops": sum(pairs) * H * G * 4 * D}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _tables(case, gen, device):
    end, new = _sizes(case)
    page = case["page"]
    most = max(1, max(-(-e // page) for e in end))
    need = [-(-e // page) for e in end]
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=gen).tolist()
    table, at = torch.zeros((case["batch"], most), dtype=torch.int32), 0
    for i, k in enumerate(need):
        table[i, :k] = torch.tensor(perm[at:at + k], dtype=torch.int32)
        at += k
    starts = [0]
    for k in new:
        starts.append(starts[-1] + k)
    return (n_pages, table.to(device), torch.tensor(end, dtype=torch.int32, device=device),
            torch.tensor(starts, dtype=torch.int32, device=device))


def _values(rows, heads, dim, gen, dtype, device, offsets):
    """Activations of `heads` heads: each channel has its own spread, some (as keys do) an offset."""
    spread = torch.exp(torch.empty((heads, dim), device=device).uniform_(math.log(0.2), math.log(3.0), generator=gen))
    x = torch.randn((rows, heads, dim), generator=gen, device=device, dtype=torch.float32)
    x *= spread
    if offsets:
        far = torch.rand((heads, dim), generator=gen, device=device) < 0.1
        x += far * torch.randn((heads, dim), generator=gen, device=device) * 4.0
    return x.to(dtype)


def _inputs(case, seed, device="cuda"):
    """What the definition is given: the tokens' keys and values by sequence, the queries, the tables."""
    gen = torch.Generator(device=device).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    H, G, D, dt = case["kv_heads"], case["q_per_kv"], case["head_dim"], _TYPES[case["dtype"]]
    end, new = _sizes(case)
    d = {"tables": _tables(case, host, device)}
    held = end if case["op"] != "write" else new         # rows whose keys and values are made
    rows = sum(held)
    d["k"] = _values(rows, H, D, gen, dt, device, True)
    d["v"] = _values(rows, H, D, gen, dt, device, False)
    if case["op"] in ("decode", "prompt"):
        n = sum(new)
        # the queries stand in the rows of one fused projection, as a model's do
        fused = torch.randn((n, (G + 2) * H * D), generator=gen, device=device, dtype=torch.float32).to(dt)
        d["q"] = fused[:, :G * H * D].view(n, G * H, D)
        if case["op"] == "decode":
            d["q"] = d["q"].view(case["batch"], case["new"], G * H, D)
    return d


def _slots(ends, counts, table, page):
    """Pool row of each of the last `counts` positions of every sequence, in order (device tensors)."""
    seq = torch.repeat_interleave(torch.arange(len(counts), device=table.device), counts)
    first = torch.cumsum(counts, 0) - counts
    pos = torch.arange(len(seq), device=table.device) - first[seq] + (ends - counts)[seq]
    return table[seq, pos // page].long() * page + pos % page


def prepare(case, seed):
    d = _inputs(case, seed)
    n_pages, table, end, starts = d["tables"]
    page, H, D, group = case["page"], case["kv_heads"], case["head_dim"], case["group"]
    s = {"case": case, "table": table, "end": end, "starts": starts, "scale": 1.0 / math.sqrt(D)}
    s["rows"] = sum(_sizes(case)[1])
    if case["op"] == "write":
        s["k"], s["v"] = d["k"], d["v"]
    elif "q" in d:
        s["q"] = d["q"]
    if own:
        import delta_quantized_kv_b200 as dkv
        s["cache"] = dkv.Kv4Cache(n_pages, H, head_dim=D, page_size=page, group=group)
        if case["op"] != "write":
            held = torch.cat([torch.zeros_like(end[:1]), torch.cumsum(end, 0, dtype=torch.int32)])
            s["cache"].append(d["k"], d["v"], table, end, held)
        return s
    NB = D // group
    for t in ("k", "v"):     # the same cache, unpacked: codes, zero points and scales of every pool row
        s[t + "_code"] = torch.zeros((n_pages * page, H, NB, group), dtype=torch.uint8, device="cuda")
        s[t + "_zero"] = torch.zeros((n_pages * page, H, NB, 1), dtype=torch.uint8, device="cuda")
        s[t + "_scale"] = torch.zeros((n_pages * page, H, NB, 1), dtype=torch.float16, device="cuda")
    if case["op"] != "write":
        _plain_write(s, d["k"], d["v"], _slots(end.long(), end.long(), table, page))
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _plain_quantise(x, group):
    x = torch.nan_to_num(x.float(), nan=0.0).clamp(-32768.0, 32768.0)
    x = x.view(x.shape[0], x.shape[1], -1, group)
    hi = x.amax(-1, keepdim=True).clamp_min(0.0)
    lo = x.amin(-1, keepdim=True).clamp_max(0.0)
    r = (hi - lo) * torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)
    up = ((r.view(torch.int32) + 0x1FFFF) & ~0x1FFFF).view(torch.float32)
    s = torch.where(r < 2.0 ** -14, torch.ceil(r * 2.0 ** 20) * 2.0 ** -20, up)
    div = torch.where(s > 0, s, torch.ones_like(s))
    zero = torch.round(-lo / div).clamp_max(15.0)
    code = (torch.round(x / div) + zero).clamp(0.0, 15.0)
    none = s == 0
    return code.masked_fill(none, 0.0).to(torch.uint8), zero.masked_fill(none, 0.0).to(torch.uint8), s.half()


def _plain_write(s, k, v, slots):
    group = s["case"]["group"]
    s["k_code"][slots], s["k_zero"][slots], s["k_scale"][slots] = _plain_quantise(k, group)
    s["v_code"][slots], s["v_zero"][slots], s["v_scale"][slots] = _plain_quantise(v, group)


def _plain_read(s, t, rows):
    """Pool rows `rows` of tensor t as fp32 [..., kv heads, head_dim]."""
    x = (s[t + "_code"][rows].float() - s[t + "_zero"][rows].float()) * s[t + "_scale"][rows].float()
    return x.flatten(-2)


def _plain_attention(s, q, asked):
    """q: [batch, m, heads, dim], m the most queries of a sequence; query i of sequence b, for i < asked[b], is
    that of position end[b] - asked[b] + i."""
    case, table, end = s["case"], s["table"], s["end"].long()
    B, m, Hq, D = q.shape
    H, page = case["kv_heads"], case["page"]
    L = table.shape[1] * page
    rows = (table.long()[:, :, None] * page + torch.arange(page, device=q.device)).view(B, L)
    k = _plain_read(s, "k", rows).permute(0, 2, 3, 1)                       # B H D L
    v = _plain_read(s, "v", rows).transpose(1, 2)                           # B H L D
    q = q.float().view(B, m, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    x = (q @ k) * s["scale"]                                                # B H (m G) L
    at = end[:, None] - asked[:, None] + torch.arange(m, device=q.device)   # B m: the queries' positions
    pos = torch.arange(L, device=q.device)
    seen = (pos <= at[..., None]) & (pos < end[:, None, None])
    if case["window"]:
        seen &= pos > at[..., None] - case["window"]
    seen = seen[:, None, :, None, :].expand(B, 1, m, Hq // H, L).reshape(B, 1, -1, L)
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = x.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = (w @ v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top).squeeze(-1)
    o = o.view(B, H, m, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, m, Hq, D)
    return o, lse.view(B, H, m, Hq // H).permute(0, 2, 1, 3).reshape(B, m, Hq)


def run(s):
    case = s["case"]
    dt, op = _TYPES[case["dtype"]], case["op"]
    if own:
        c = s["cache"]
        if op == "write":
            c.append(s["k"], s["v"], s["table"], s["end"], s["starts"])
        if op in ("write", "read"):
            k, v = c.read(s["rows"], s["table"], s["end"], s["starts"], dtype=dt)
            return {"k": k, "v": v}
        kw = {"window": case["window"], "return_lse": case["lse"]}
        if op == "decode":
            r = c.decode_attn(s["q"], s["scale"], s["table"], s["end"], **kw)
        else:
            r = c.prompt_attn(s["q"], s["scale"], s["table"], s["end"], s["starts"], **kw)
        return {"out": r[0], "lse": r[1]} if case["lse"] else {"out": r}
    new = (s["starts"][1:] - s["starts"][:-1]).long()
    if op in ("write", "read"):
        slots = _slots(s["end"].long(), new, s["table"], case["page"])
        if op == "write":
            _plain_write(s, s["k"], s["v"], slots)
        return {"k": _plain_read(s, "k", slots).to(dt), "v": _plain_read(s, "v", slots).to(dt)}
    q = s["q"]
    if op == "decode":
        o, lse = _plain_attention(s, q, new)
    else:   # padded to the longest chunk and back
        seq = torch.repeat_interleave(torch.arange(case["batch"], device=q.device), new)
        i = torch.arange(len(seq), device=q.device) - s["starts"][:-1].long()[seq]
        padded = q.new_zeros((case["batch"], case["new"]) + q.shape[1:])
        padded[seq, i] = q
        o, lse = _plain_attention(s, padded, new)
        o, lse = o[seq, i], lse[seq, i]
    return {"out": o.to(dt), "lse": lse} if case["lse"] else {"out": o.to(dt)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_values(x, group):
    """The values held for tokens x [n, heads, dim]: the rule's fp32 roundings, taken of 64-bit results."""
    def f32(y):
        return y.to(torch.float32).double()

    y = x.double()
    y = torch.where(torch.isnan(y), torch.zeros_like(y), y)
    y = torch.minimum(torch.maximum(y, y.new_tensor(-32768.0)), y.new_tensor(32768.0))
    y = y.unflatten(-1, (-1, group))
    zero = y.new_zeros(())
    hi = torch.maximum(y.max(dim=-1, keepdim=True).values, zero)
    lo = torch.minimum(y.min(dim=-1, keepdim=True).values, zero)
    r = f32(f32(hi - lo) * f32(y.new_tensor(1.0) / 15.0))
    e = torch.clamp(torch.frexp(r)[1] - 7, min=-20)      # 7 bits: multiples of 2^e
    s = torch.ldexp(torch.ceil(torch.ldexp(r, -e)), e)
    d = torch.where(s > 0, s, torch.ones_like(s))
    z = torch.minimum(torch.round(f32(-lo / d)), y.new_tensor(15.0))
    c = torch.minimum(torch.maximum(torch.round(f32(y / d)) + z, zero), y.new_tensor(15.0))
    return ((c - z) * s).flatten(-2)


def exact(case, seed):
    d = _inputs(case, seed)
    end, new = _sizes(case)
    group = case["group"]
    if case["op"] == "write":
        return {"k": _exact_values(d["k"], group), "v": _exact_values(d["v"], group)}
    first = [0]
    for e in end:
        first.append(first[-1] + e)
    if case["op"] == "read":
        at = [torch.arange(first[i] + e - n, first[i] + e) for i, (e, n) in enumerate(zip(end, new))]
        at = torch.cat(at).to(d["k"].device)
        return {"k": _exact_values(d["k"][at], group), "v": _exact_values(d["v"][at], group)}
    H, G, D, w = case["kv_heads"], case["q_per_kv"], case["head_dim"], case["window"]
    q = d["q"].reshape(-1, H * G, D)
    out = torch.zeros((q.shape[0], H * G, D), dtype=torch.float64, device=q.device)
    lse = torch.full((q.shape[0], H * G), -math.inf, dtype=torch.float64, device=q.device)
    row = 0
    for b in range(case["batch"]):
        e, n = end[b], new[b]
        if min(e, n) > 0:
            ks = _exact_values(d["k"][first[b]:first[b + 1]], group)
            vs = _exact_values(d["v"][first[b]:first[b + 1]], group)
            for i in range(0, n, 2048):
                k = min(2048, n - i)
                at = torch.arange(e - n + i, e - n + i + k, device=q.device)[:, None]
                pos = torch.arange(e, device=q.device)[None]
                off = (pos > at) | (pos <= at - w) if w else pos > at
                for h in range(H * G):
                    x = q[row + i:row + i + k, h].double() @ ks[:, h // G].T / math.sqrt(D)
                    x = x.masked_fill(off, -math.inf)
                    lse[row + i:row + i + k, h] = torch.logsumexp(x, -1)
                    out[row + i:row + i + k, h] = torch.softmax(x, -1) @ vs[:, h // G]
        row += n
    return {"out": out.reshape(d["q"].shape), "lse": lse.view(d["q"].shape[:-1])} if case["lse"] else \
        {"out": out.reshape(d["q"].shape)}
