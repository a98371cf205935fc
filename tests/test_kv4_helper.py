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
