"""CPU checks of the paged 4-bit cache's sources: properties that no run on a
GPU that works shows."""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "delta_quantized_kv_b200" / "csrc"


def code(name):
    """A source file without its comments."""
    s = (CSRC / name).read_text()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", s, flags=re.S))


@pytest.mark.parametrize("name", ["kv4_common.cuh", "kv4_write.cu", "kv4_decode.cu", "kv4_prompt.cu"])
def test_a_warp_gives_up_a_wait_together(name):
    """Each lane of a bounded wait has its own clock.  Lanes that differ about
    the outcome would leave the others in shuffles and votes of the whole warp,
    which wait for all of them."""
    s = code(name)
    waits = [m.start() for m in re.finditer(r"\bmbar_wait_bounded\(", s)]
    vote = "__all_sync(0xffffffffu, "
    assert all(s[:i].endswith(vote) for i in waits)
    assert bool(waits) == (name == "kv4_common.cuh")


@pytest.mark.parametrize("name", ["dkv_api.cu", "kv4_api.cu"])
def test_status_words_are_cleared_of_what_was_read(name):
    """Both caches' status reads go through the one that clears bits atomically."""
    s = code(name)
    body = s[s.index("get_device_status("):]
    body = body[:body.index("\n}\n")]
    assert "take_status(" in body and "Memset" not in body and "Memcpy" not in body
    assert "atomicAnd(word, ~bits)" in code("status.cu")


def test_every_source_is_built():
    from delta_quantized_kv_b200 import build
    assert sorted(p.name for p in CSRC.glob("*.cu")) == sorted(build.SOURCES)
    assert sorted(p.name for p in CSRC.iterdir() if p.suffix in (".cuh", ".h")) == sorted(build.HEADERS)
