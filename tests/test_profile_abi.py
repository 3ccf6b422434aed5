"""hisa_profile_read keeps the number of entries that programs built with the
first header gave it room for; hisa_profile_read_n writes what it is asked."""
import ctypes
import os
import re

import hierarchical_top_indexer_b200 as hisa
from tests.test_abi import HEADER

FIRST_HEADER = 12    # phases before hisa_rope, hisa_cache_* and hisa_block_attn


def _arrays(n, fill=77):
    return (ctypes.c_float * n)(*[fill] * n), (ctypes.c_int * n)(*[fill] * n)


def test_profile_read_writes_the_first_headers_entries():
    ms, count = _arrays(FIRST_HEADER + 8)
    assert hisa.lib().hisa_profile_read(ms, count, 1) == hisa.HISA_OK
    for a in (ms, count):
        assert list(a[:FIRST_HEADER]) == [0] * FIRST_HEADER and list(a[FIRST_HEADER:]) == [77] * 8
    assert hisa.lib().hisa_profile_read(None, None, 0) == hisa.HISA_OK


def test_profile_read_n_writes_n_entries():
    for n in (0, 1, FIRST_HEADER, len(hisa.PHASES), len(hisa.PHASES) + 3):
        ms, count = _arrays(n + 2)
        assert hisa.lib().hisa_profile_read_n(ms, count, n, 0) == hisa.HISA_OK
        for a in (ms, count):
            assert list(a) == [0] * n + [77] * 2
    assert hisa.lib().hisa_profile_read_n(None, None, -1, 0) == hisa.HISA_E_INVAL
    assert tuple(hisa.hisa_profile_read()) == hisa.PHASES


def test_the_headers_numbers():
    text = open(os.path.join(HEADER)).read()
    number = lambda name: int(re.search(rf"\b{name} = (\d+)", text).group(1))  # noqa: E731
    assert number("HISA_NUM_PHASES") == FIRST_HEADER == number("HISA_PHASE_ROPE")
    assert number("HISA_NUM_ALL_PHASES") == len(hisa.PHASES) == number("HISA_PHASE_BLOCK_ATTN") + 1
