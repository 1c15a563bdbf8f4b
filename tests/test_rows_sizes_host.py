"""Refusals of the calls on rows of any number at the ends of their ranges, on the
host."""
import pytest

import speculative_decoding_verification_softmax_gb300 as sv
from tests.test_cache_host import P
from tests.test_rows_host import map_rows


@pytest.fixture(scope="module")
def L():
    sv.build()
    return sv.lib()


@pytest.mark.parametrize("bad,code", [
    (dict(request=None), "NULL"), (dict(position=None), "NULL"), (dict(slot=None), "NULL"), (dict(first=P + 2), "ALIGN"),
    (dict(request=P + 2), "ALIGN"), (dict(position=P + 1), "ALIGN"), (dict(slot=P + 4), "ALIGN"), (dict(rows=-1), "SHAPE")])
def test_a_map_of_no_requests_looks_at_its_arrays(L, bad, code):
    assert map_rows(L, B=0, table=None, num=None, ref=None, len=None, new=None, status=None, **bad) == \
        getattr(sv, "ERR_" + code)


def test_rows_whose_sums_could_not_be_told_apart(L):
    """Sums of lengths stop at 2^30 - 1: the arrays have to be smaller, so that such a sum lies behind them."""
    assert map_rows(L, rows=0x3fffffff) == sv.ERR_SHAPE
    assert map_rows(L, rows=0x3ffffffe, bytes=16) == sv.ERR_WORKSPACE
