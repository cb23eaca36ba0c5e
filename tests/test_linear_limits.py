"""Limits of the calls of linear attention and tables that are refused before any launch."""
import ctypes

import pytest

from paged_kv_cache_258_gb300 import pkv

PTR, NULL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0)


@pytest.mark.parametrize("n", [0, 3])
def test_more_tokens_than_the_tables_sums_hold_are_refused(n):
    """A sum past 2^31 - 1 counts as 2^31 - 1, which must not fit."""
    got = pkv.lib().pkv_extend_tables(9, PTR, 4, PTR, PTR, 4, PTR, PTR, n, PTR, 2 ** 31 - 1, PTR, PTR, PTR, NULL)
    assert got == pkv.PKV_ERR_UNSUPPORTED
