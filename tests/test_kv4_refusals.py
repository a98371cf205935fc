"""CPU check of the paged 4-bit cache's limits on rows: index sums of the
kernels stay in 32 bits."""
import pytest

from test_kv4_host import _calls, _seqs, dkv  # noqa: F401


@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 1023])
def test_rows_next_to_the_end_of_32_bits(dkv, n):  # noqa: F811
    # (uniform rows as well as ragged ones; one sequence, so that any count divides)
    for starts in (1 << 20, None):
        calls = _calls(dkv, seqs=_seqs(dkv, batch=1, starts=starts), n=n)
        for f in ("append", "append_v", "read", "prompt"):
            assert calls[f]() == dkv.DKV_ECAPACITY, f
