"""What the page calls refuse for the number of pages, before anything is launched."""
import ctypes

import pytest

from sparse_kv_long_sfi_gb300 import _abi

A = 4096  # an aligned address; nothing is read


@pytest.mark.parametrize("pages,status", [(2 ** 31 - 8191, 2), (2 ** 31 - 1, 2), (2 ** 31 - 8192, 3), (9, 3)])
def test_compaction_of_nearly_all_ids(pages, status):
    """Its plan walks the counts in steps of 8192: past 2^31 they would wrap. (3: no workspace is given.)"""
    from sparse_kv_long_sfi_gb300 import build
    build.build()
    m = _abi.sfi_page_map(A, A, A, 3, 4, pages, 16)
    q = _abi.sfi_page_pools(A, 1, 256, pages)
    assert _abi.lib().sfi_page_compact(ctypes.byref(m), ctypes.byref(q), 2 * A, 2 * A, A, None, 0, None, None) == status
