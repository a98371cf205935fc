"""CPU checks of the Kv4Cache helper (and of Cache's constructor): what they do with streams,
devices and arguments, on a torch.cuda and a library that only take notes."""
import contextlib
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture
def fake(monkeypatch):
    """torch.cuda with devices 0 and 1 and notes of the stream and device that
    each allocation and each launch happened on."""
    from delta_quantized_kv_b200 import build
    build.build()
    import delta_quantized_kv_b200 as dkv
    dkv.load()
    f = SimpleNamespace(dkv=dkv, device=0, stream="default", notes=[], side=SimpleNamespace(
        device=torch.device("cuda", 0), cuda_stream=77))

    @contextlib.contextmanager
    def on(device, stream):
        was = f.device, f.stream
        f.device, f.stream = device, stream
        yield
        f.device, f.stream = was

    def empty(*size, device=None, **kw):
        f.notes.append(("empty", f.device, f.stream))
        return real(*size, **kw)

    def init(desc, pool, n_pages, status, stream=None):
        f.notes.append(("init", f.device, f.stream if stream is None else stream))
        return dkv.dkv_kv4_pool()

    real = torch.empty
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: f.device)
    monkeypatch.setattr(torch.cuda, "device", lambda d: on(torch.device(d).index, f.stream))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: on(s.device.index, s))
    monkeypatch.setattr(dkv, "dkv_kv4_init", init)
    return f


def test_the_pool_is_taken_on_the_stream_that_zeroes_it(fake):
    fake.dkv.Kv4Cache(3, 2, device="cuda:0", stream=fake.side)
    assert [n[0] for n in fake.notes] == ["empty", "empty", "init"]
    assert all(n[1:] == (0, fake.side) for n in fake.notes)
    assert (fake.device, fake.stream) == (0, "default")
    fake.notes.clear()
    fake.dkv.Kv4Cache(3, 2, device="cuda")
    assert all(n[1:] == (0, "default") for n in fake.notes)
    fake.notes.clear()
    fake.dkv.Kv4Cache(3, 2, device="cuda:1")
    assert all(n[1:] == (1, "default") for n in fake.notes)


def test_the_delta_caches_memory_too(fake, monkeypatch):
    def init(desc, base, nbytes, stream=None):
        fake.notes.append(("init", fake.device, fake.stream if stream is None else stream))
        return fake.dkv.dkv_cache()

    monkeypatch.setattr(fake.dkv, "dkv_cache_init", init)
    for stream in (fake.side, None):
        fake.notes.clear()
        fake.dkv.Cache(1, 2, 64, device="cuda", stream=stream)
        assert [n[0] for n in fake.notes] == ["empty", "init"]
        assert all(n[1:] == (0, stream or "default") for n in fake.notes)


def test_a_fault_reported_while_the_status_is_read_is_not_lost(fake, monkeypatch):
    word = [0x1]

    def read(*_):                     # another stream reports 0x10 right behind the read
        seen = word[0]
        word[0] |= 0x10
        return seen

    def library(pool, stream=None):   # clears what it read
        seen = read()
        word[0] &= ~seen
        return seen

    cache = fake.dkv.Kv4Cache(3, 2, device="cuda:0")
    cache._stream = lambda index: 0
    cache.status = SimpleNamespace(item=read, zero_=lambda: word.__setitem__(0, 0))
    monkeypatch.setattr(fake.dkv, "dkv_kv4_get_device_status", library, raising=False)
    assert cache.device_status() == 0x1
    assert cache.device_status() & 0x10


def test_refused_status_reads(fake):
    import ctypes
    d, lib, b = fake.dkv, fake.dkv.load(), ctypes.byref
    word, P = ctypes.c_int32(5), 1 << 20
    desc = d.dkv_kv4_desc(2, 128, 32, 64)
    nb = d.dkv_kv4_page_bytes(desc)
    for pool, out, want in ((None, b(word), d.DKV_EINVAL), (d.dkv_kv4_pool(desc, P, 4, nb, P), None, d.DKV_EINVAL),
                            (d.dkv_kv4_pool(desc, P, 4, nb, None), b(word), d.DKV_EINVAL),
                            (d.dkv_kv4_pool(desc, P, 4, nb, P + 2), b(word), d.DKV_EALIGN)):
        assert lib.dkv_kv4_get_device_status(None if pool is None else b(pool), out, 0) == want
        assert word.value == 5


def test_a_missing_table_or_length_is_refused(fake):
    cache = fake.dkv.Kv4Cache(3, 2, device="cuda:0")
    q = torch.zeros(1, 4, 128, dtype=torch.float16)
    on = SimpleNamespace(get_device=lambda: 0, dim=lambda: 2, dtype=torch.int32, is_contiguous=lambda: True, shape=(1, 3))
    for table in (None, on):
        for call in (lambda: cache.read(2, table, None), lambda: cache.decode_attn(q, 0.1, table, None),
                     lambda: cache.prompt_attn(q, 0.1, table, None)):
            with pytest.raises(ValueError, match="seq_lens" if table else "block_table"):
                call()


def test_a_stream_of_another_device_is_refused(fake):
    """A call on it would go to a stream that the caller does not know."""
    cache = fake.dkv.Kv4Cache(3, 2, device="cuda:0")
    other = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=78)
    q = torch.zeros(1, 4, 128, dtype=torch.float16)
    for call in (lambda: cache.append(q, q, None, None, stream=other), lambda: cache.read(1, None, None, stream=other),
                 lambda: cache.decode_attn(q, 0.1, None, None, stream=other),
                 lambda: cache.prompt_attn(q, 0.1, None, None, stream=other),
                 lambda: cache.device_status(stream=other),
                 lambda: fake.dkv.Kv4Cache(3, 2, device="cuda:0", stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert (fake.device, fake.stream) == (0, "default")


@pytest.fixture
def on_cpu(fake):
    """A cache whose tensors are the CPU's, with a library that notes the
    arguments of its calls."""
    cache = fake.dkv.Kv4Cache(3, 2, device="cuda:0")
    cache.device, cache._index, fake.device = torch.device("cpu"), -1, -1
    cache._stream = lambda index: 0
    cache.calls = []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                cache.calls.append((name, args))
                return 64 if name.endswith("_bytes") else 0
            return call

    cache._lib = Library()
    cache.table, cache.lens = torch.zeros((2, 3), dtype=torch.int32), torch.tensor([5, 7], dtype=torch.int32)
    return cache


def test_types_that_read_does_not_give_are_refused(on_cpu):
    c = on_cpu
    two = (torch.zeros(2, 2, 128, dtype=torch.float64), torch.zeros(2, 2, 128, dtype=torch.float64))
    for kw in (dict(dtype=torch.float64), dict(dtype=torch.int8), dict(out=two), dict(out=two, dtype=torch.float64)):
        for n in (2, 0):
            with pytest.raises(ValueError):
                c.read(n, c.table, c.lens, **{**kw, **({"out": tuple(x[:n] for x in two)} if "out" in kw else {})})
    assert not c.calls
    assert c.read(2, c.table, c.lens)[0].dtype == torch.float16
    assert c.read(0, c.table, c.lens, dtype=torch.bfloat16)[1].dtype == torch.bfloat16


def test_numbers_past_32_bits_are_refused_or_kept(on_cpu, fake):
    """The library's counts and windows have 32 bits; what passes them must not
    come out as something else."""
    import ctypes
    c = on_cpu
    q = torch.zeros(2, 4, 128, dtype=torch.float16)
    for window in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63):
        for f in (c.decode_attn, c.prompt_attn):
            c.calls.clear()
            f(q, 0.1, c.table, c.lens, window=window)
            got = c.calls[-1][1][9]                     # past every position: as none
            assert ctypes.c_int32(got).value == got and got > 1 << 30
    for window in (-1, -2 ** 31, -2 ** 32, -2 ** 32 - 5):
        for f in (c.decode_attn, c.prompt_attn):
            c.calls.clear()
            f(q, 0.1, c.table, c.lens, window=window)   # (the library refuses it)
            assert ctypes.c_int32(c.calls[-1][1][9]).value < 0
    c.calls.clear()
    k = torch.zeros((1, 2, 128), dtype=torch.float16).expand(2 ** 32 + 2, 2, 128)
    table = SimpleNamespace(get_device=lambda: -1, dim=lambda: 2, dtype=torch.int32, is_contiguous=lambda: True,
                            shape=(2, 2 ** 32 + 3), data_ptr=lambda: 256)
    with pytest.raises(ValueError):
        c.append(k, k, c.table, c.lens)
    with pytest.raises(ValueError):
        c.append(q[:, :2], q[:, :2], table, c.lens)
    for bad in (dict(n_kv_heads=2 ** 32 + 2), dict(head_dim=128 - 2 ** 32), dict(group=2 ** 32 + 32),
                dict(page_size=2 ** 32 + 64)):
        with pytest.raises(fake.dkv.DkvError):
            fake.dkv.Kv4Cache(3, **{"n_kv_heads": 2, "device": "cuda:0", **bad})
    assert not c.calls

