"""The calls on rows of any number refuse bad arguments on the host, before the
device is touched."""
import pytest
import torch

import speculative_decoding_verification_softmax_gb300 as sv
from tests.test_cache_host import BAD_CACHES, P, cache


@pytest.fixture(scope="module")
def L():
    sv.build()
    return sv.lib()


def append(L, c=None, **kw):
    d = dict(q=P, qrs=512, qhs=64, k=P, v=P, krs=128, khs=64, vrs=128, vhs=64, dt=sv.BF16, heads=8, cache=c or cache(),
             position=P, slot=P, rows=20, turns=P, rotary=64, interleaved=0, mscale=1.0, out=P, ws=P, bytes=256,
             stream=None)
    d.update(kw)
    return L.spec_append_rows(*d.values())


def map_rows(L, **kw):
    d = dict(table=P, num=P, ref=P, pages=100, len=P, new=P, B=4, slots=10, page=16, rows=20, first=P, request=P,
             position=P, slot=P, status=P, ws=P, bytes=256, stream=None)
    d.update(kw)
    return L.spec_map_rows(*d.values())


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches(L, bad, code):
    assert append(L, cache(**bad)) == getattr(sv, "ERR_" + code)


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), "SHAPE"), (dict(heads=-1), "SHAPE"), (dict(heads=65536), "SHAPE"), (dict(dt=sv.E4M3), "SHAPE"),
    (dict(dt=sv.F16), "SHAPE"), (dict(dt=sv.F32), "SHAPE"), (dict(rotary=-2), "SHAPE"), (dict(rotary=66), "SHAPE"),
    (dict(rotary=7), "SHAPE"), (dict(mscale=float("nan")), "SHAPE"), (dict(mscale=float("inf")), "SHAPE"),
    (dict(q=None), "NULL"), (dict(out=None), "NULL"), (dict(k=None), "NULL"), (dict(v=None), "NULL"),
    (dict(position=None), "NULL"), (dict(slot=None), "NULL"), (dict(turns=None), "NULL"), (dict(ws=None), "NULL"),
    (dict(q=P + 2), "ALIGN"), (dict(k=P + 8), "ALIGN"), (dict(v=P + 8), "ALIGN"), (dict(out=P + 8), "ALIGN"),
    (dict(ws=P + 8), "ALIGN"), (dict(position=P + 2), "ALIGN"), (dict(slot=P + 4), "ALIGN"), (dict(turns=P + 4), "ALIGN"),
    (dict(qrs=1), "ALIGN"), (dict(khs=4), "ALIGN"), (dict(vrs=4), "ALIGN"), (dict(bytes=16), "WORKSPACE")])
def test_append_refusals(L, bad, code):
    assert append(L, **bad) == getattr(sv, "ERR_" + code)


def test_e4m3_cache_needs_16_bit_rows(L):
    c = cache(dt=sv.E4M3)
    assert append(L, c, dt=sv.F32) == sv.ERR_SHAPE
    assert append(L, c, bytes=0) == sv.ERR_WORKSPACE


def test_without_queries(L):
    """q and out_q are not looked at: the refusal is the next one's."""
    assert append(L, heads=0, q=None, out=None, k=None) == sv.ERR_NULL
    assert append(L, heads=0, q=P + 2, qrs=1, out=P + 2, bytes=16) == sv.ERR_WORKSPACE


def test_no_rows_are_a_no_op(L):
    assert append(L, rows=0, q=None, k=None, position=None, ws=None) == sv.OK
    assert map_rows(L, B=0, table=None, first=None) == sv.OK


@pytest.mark.parametrize("bad,code", [
    (dict(B=-1), "SHAPE"), (dict(B=4097), "SHAPE"), (dict(slots=0), "SHAPE"), (dict(pages=0), "SHAPE"),
    (dict(page=0), "SHAPE"), (dict(rows=-1), "SHAPE"), (dict(rows=0x40000000), "SHAPE"), (dict(table=None), "NULL"),
    (dict(num=None), "NULL"), (dict(ref=None), "NULL"), (dict(len=None), "NULL"), (dict(new=None), "NULL"),
    (dict(first=None), "NULL"), (dict(request=None), "NULL"), (dict(position=None), "NULL"), (dict(slot=None), "NULL"),
    (dict(status=None), "NULL"), (dict(ws=None), "NULL"), (dict(table=P + 2), "ALIGN"), (dict(new=P + 1), "ALIGN"),
    (dict(first=P + 1), "ALIGN"), (dict(request=P + 1), "ALIGN"), (dict(position=P + 1), "ALIGN"),
    (dict(slot=P + 4), "ALIGN"), (dict(status=P + 1), "ALIGN"), (dict(ws=P + 8), "ALIGN"), (dict(bytes=16), "WORKSPACE")])
def test_map_refusals(L, bad, code):
    assert map_rows(L, **bad) == getattr(sv, "ERR_" + code)


def test_binding_refusals():
    z = torch.zeros
    k, pos, slot = z(3, 2, 64, dtype=torch.bfloat16), z(3, dtype=torch.int32), z(3, dtype=torch.int64)
    K = z(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.append_rows(None, k, k, K, K, pos, slot)                           # host tensors
    with pytest.raises(ValueError):
        sv.append_rows(None, k[None], k[None], K, K, pos, slot)
    with pytest.raises(TypeError):
        sv.append_rows(None, k.to(torch.float64), k, K, K, pos, slot)
    with pytest.raises(ValueError):
        sv.map_rows(z(2, 3, dtype=torch.int32), z(2, dtype=torch.int32), z(9, dtype=torch.int32),
                    z(2, dtype=torch.int32), z(2, dtype=torch.int32), rows=5, page_size=16)
