"""Host-side refusals of d2f_page_map_flags (no GPU: refused before anything is enqueued)."""
import ctypes

import pytest

from block_causal_kv_gb300 import d2f

P = ctypes.c_void_p(16)  # an aligned pointer that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return d2f.load()


@pytest.mark.parametrize("flags,batch,status", [(2, 2, 1), (0x80000001, 2, 1), (1, -1, 1),
                                                (1, 16385, 2)])
def test_page_map_flags_refusals(lib, flags, batch, status):
    assert lib.d2f_page_map_flags(batch, 16, 4, 32, 2, *[P] * 14, flags, None, None) == status
    assert lib.d2f_last_error_string().decode()


@pytest.mark.parametrize("null", range(14))
def test_page_map_flags_refuses_null_pointers(lib, null):
    ptr = [None if i == null else P for i in range(14)]
    assert lib.d2f_page_map_flags(2, 16, 4, 32, 2, *ptr, d2f.PAGE_MAP_FRESH, None, None) == 1
