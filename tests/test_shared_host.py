"""The calls for batches that share prefixes refuse bad arguments on the host,
before the device is touched."""
import pytest
import torch

import speculative_decoding_verification_softmax_gb300 as sv
from tests._share_model import groups
from tests.test_cache_host import BAD_CACHES, BIG, P, cache


@pytest.fixture(scope="module")
def L():
    sv.build()
    return sv.lib()


def plan(L, **kw):
    d = dict(table=P, slots=10, page=16, len=P, ell=None, row=None, rows=20, B=4, gamma=4, least=256, leader=P, shared=P,
             plan=P, bytes=BIG, stream=None)
    d.update(kw)
    return L.spec_share_plan(*d.values())


def attend(L, c=None, **kw):
    d = dict(q=P, rs=512, hs=64, dt=sv.BF16, heads=8, cache=c or cache(), table=P, slots=10, plan=P, plan_bytes=BIG,
             rows=20, B=4, gamma=4, scale=0.1, out=P, lse=None, ws=P, bytes=BIG, stream=None)
    d.update(kw)
    return L.spec_attend_shared(*d.values())


ALIKE = [(dict(B=-1), "SHAPE"), (dict(B=4097), "SHAPE"), (dict(slots=0), "SHAPE"), (dict(gamma=-1), "SHAPE"),
         (dict(gamma=33), "SHAPE"), (dict(rows=-1), "SHAPE"), (dict(table=None), "NULL"), (dict(table=P + 2), "ALIGN"),
         (dict(plan=None), "NULL"), (dict(plan=P + 8), "ALIGN"), (dict(bytes=16), "WORKSPACE")]


@pytest.mark.parametrize("bad,code", ALIKE + [
    (dict(page=0), "SHAPE"), (dict(least=-1), "SHAPE"), (dict(rows=19), "SHAPE"), (dict(len=None), "NULL"),
    (dict(leader=None), "NULL"), (dict(shared=None), "NULL"), (dict(len=P + 1), "ALIGN"), (dict(ell=P + 1), "ALIGN"),
    (dict(row=P + 1), "ALIGN"), (dict(leader=P + 1), "ALIGN"), (dict(shared=P + 2), "ALIGN")])
def test_plan_refusals(L, bad, code):
    assert plan(L, **bad) == getattr(sv, "ERR_" + code)


@pytest.mark.parametrize("bad,code", ALIKE + [
    (dict(heads=0), "SHAPE"), (dict(heads=7), "SHAPE"), (dict(dt=sv.E4M3), "SHAPE"), (dict(dt=sv.F16), "SHAPE"),
    (dict(dt=sv.F32), "SHAPE"), (dict(scale=float("nan")), "SHAPE"), (dict(scale=float("inf")), "SHAPE"),
    (dict(rows=1 << 30), "SHAPE"), (dict(q=None), "NULL"), (dict(out=None), "NULL"), (dict(ws=None), "NULL"),
    (dict(q=P + 2), "ALIGN"), (dict(out=P + 8), "ALIGN"), (dict(ws=P + 8), "ALIGN"), (dict(rs=4), "ALIGN"),
    (dict(hs=60), "ALIGN"), (dict(lse=P + 2), "ALIGN"), (dict(plan_bytes=256), "WORKSPACE")])
def test_attend_refusals(L, bad, code):
    assert attend(L, **bad) == getattr(sv, "ERR_" + code)


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches(L, bad, code):
    assert attend(L, cache(**bad)) == getattr(sv, "ERR_" + code)


def test_e4m3_cache_needs_16_bit_rows(L):
    assert attend(L, cache(dt=sv.E4M3), dt=sv.F32) == sv.ERR_SHAPE
    assert attend(L, cache(dt=sv.E4M3), bytes=0) == sv.ERR_WORKSPACE


def test_empty_batches_are_no_ops(L):
    assert plan(L, B=0, table=None, plan=None, len=None) == sv.OK
    assert attend(L, B=0, q=None, plan=None, ws=None) == sv.OK
    assert attend(L, rows=0, q=None, plan=None, ws=None) == sv.OK


def test_sizes(L):
    # header, items, list, kinds; each rounded to 256 bytes
    assert L.spec_share_plan_bytes(4, 4, 20) == 256 + 256 + 256 + 256
    assert L.spec_share_plan_bytes(4097, 4, 20) == L.spec_share_plan_bytes(4, 33, 20) == 0
    assert L.spec_share_plan_bytes(4, 4, -1) == 0
    n = L.spec_attend_shared_workspace_bytes(64, 16, 1088, 32, 8, 128)
    assert n >= 2 * 1088 * 32 * (128 * 4 + 16)
    assert L.spec_attend_shared_workspace_bytes(64, 16, 1088, 32, 7, 128) == 0
    assert L.spec_attend_shared_workspace_bytes(64, 16, 1088, 32, 8, 12) == 0
    assert L.spec_attend_shared_workspace_bytes(64, 16, 1 << 27, 32, 8, 128) == 0


def test_binding_refusals():
    table = torch.zeros(3, 4, dtype=torch.int32)
    lens = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.share_plan(table, lens, gamma=1, page_size=16)      # host tensors
    with pytest.raises(ValueError):
        k = torch.zeros(9, 16, 2, 64, dtype=torch.bfloat16)
        sv.attend_shared(torch.zeros(3, 2, 8, 64, dtype=torch.bfloat16), k, k, table, torch.zeros(1024, dtype=torch.uint8))
    with pytest.raises(ValueError):                            # packed rows need gamma
        sv.attend_shared(torch.zeros(6, 8, 64, dtype=torch.bfloat16), None, None, table, None)


def test_the_model_of_the_plan():
    # all of 0..3 share two pages, 1 and 3 one more; the head's best is the whole class
    table = [[5, 6, 1, 2], [5, 6, 7, 3], [5, 6, 4, -1], [5, 6, 7, 8], [9, 10, -1, -1]]
    lens = [16 * 4, 16 * 4, 16 * 2 + 3, 16 * 3, 16]
    assert groups(table, lens, 16, 1) == ([0, 0, 0, 0, 4], [2, 2, 2, 2, 0])
    # prefixes of two pages are too short: 0 is alone, then 1 and 3 share three
    assert groups(table, lens, 16, 48) == ([0, 1, 2, 1, 4], [0, 3, 0, 3, 0])
    assert groups(table, lens, 16, 49) == ([0, 1, 2, 3, 4], [0] * 5)
