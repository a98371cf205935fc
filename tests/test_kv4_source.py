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


def test_the_runs_test_has_the_kernels_constants():
    """test_kv4_host.py restates the formulas that cut a prompt call into runs."""
    import test_kv4_host as host
    s = code("kv4_prompt.cu")
    for name in ("TM", "TN", "COST", "MIN_TILES"):
        assert int(re.search(rf"constexpr int {name} = (\d+);", s).group(1)) == getattr(host, name)
    # and the formulas themselves, line for line
    for line in ("const int64_t k = u.full <= u.base ? 0 : min(m, (u.full - u.base) / (2 * TM));",
                 "return u.base * k + TM * k * (k + 1) + (m > k ? (m - k) * u.full : 0) + m * u.cost;",
                 "return min(u.full, u.base + 2 * TM * (m + 1)) + u.cost;",
                 "u.full = p.q.window > 0 ? (int64_t)p.G * p.q.window + 2 * TM : INT64_MAX;",
                 "u.cost = (int64_t)COST * TN * p.G;",
                 "const int64_t least = (int64_t)MIN_TILES * TN * G, n = total / least;",
                 "const int64_t each = (units - u.cost + tiles - 1) / tiles;"):
        assert line in s, line


def test_a_split_warp_that_gives_up_says_so():
    """Delta-KV's split kernel: any lane may run out of time first, so the report
    comes behind the warp's vote and not from lane 0's own clock."""
    s = code("decode.cu")
    body = s[s.index("if (!mbar_wait_bounded("):]
    body = body[:body.index("if (dead) break;")]
    assert body.index("__any_sync(0xffffffffu, dead)") < body.index("set_status(cv.header, DKV_DEV_TIMEOUT)")
