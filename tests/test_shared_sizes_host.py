"""Sizes of shared-prefix attention whose row counts would leave 32 bits, on the
host."""
import pytest

import speculative_decoding_verification_softmax_gb300 as sv
from tests.test_cache_host import cache
from tests.test_shared_host import attend


@pytest.fixture(scope="module")
def L():
    sv.build()
    return sv.lib()


def test_a_groups_rows_stay_in_31_bits(L):
    """Rows that requests name twice count twice in a group: its rows of a KV head are bounded by the batch's, not by
    the array's."""
    c = cache(kv_heads=1)
    big = dict(B=4096, gamma=32, heads=65535, rows=20)
    assert attend(L, c, **big) == sv.ERR_SHAPE
    assert L.spec_attend_shared_workspace_bytes(4096, 32, 20, 65535, 1, 64) == 0
    most = 0x7fffff00 // (4096 * 33)
    assert L.spec_attend_shared_workspace_bytes(4096, 32, 20, most, 1, 64) > 0
    assert attend(L, c, **dict(big, heads=most, bytes=16)) == sv.ERR_WORKSPACE
