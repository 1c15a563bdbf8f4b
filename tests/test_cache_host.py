"""The cache calls refuse bad arguments on the host, before the device is
touched, and the rotary tables' arithmetic."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verification_softmax_gb300 as sv

P = 0x10000   # never dereferenced: every case fails host validation, or has nothing to do
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    sv.build()
    return sv.lib()


def cache(**kw):
    d = dict(k=P, v=P, dt=sv.BF16, layers=1, pages=100, page_size=16, kv_heads=2, head_dim=64, layer_stride=64,
             page_stride=16 * 128, token_stride=128, head_stride=64, k_scale=None, v_scale=None)
    d.update(kw)
    return sv.Cache(*[d[f[0]] for f in sv.Cache._fields_])


BAD_CACHES = [(dict(dt=4), "SHAPE"), (dict(dt=-1), "SHAPE"), (dict(pages=0), "SHAPE"), (dict(page_size=0), "SHAPE"),
              (dict(layers=0), "SHAPE"), (dict(kv_heads=0), "SHAPE"), (dict(head_dim=0), "SHAPE"),
              (dict(head_dim=60), "SHAPE"), (dict(head_dim=264), "SHAPE"), (dict(dt=sv.E4M3, head_dim=72), "SHAPE"),
              (dict(k=None), "NULL"), (dict(v=None), "NULL"), (dict(k=P + 8), "ALIGN"), (dict(v=P + 2), "ALIGN"),
              (dict(page_stride=100), "ALIGN"), (dict(token_stride=4), "ALIGN"), (dict(head_stride=2), "ALIGN"),
              (dict(layer_stride=1), "ALIGN"), (dict(k_scale=P + 1), "ALIGN")]


def attend(L, c=None, **kw):
    d = dict(q=P, rs=512, hs=64, dt=sv.BF16, heads=8, cache=c or cache(), table=P, slots=10, len=P, ell=None, row=None,
             rows=20, B=4, gamma=4, scale=0.1, window=0, sinks=0, out=P, lse=None, ws=P, bytes=BIG, stream=None)
    d.update(kw)
    return L.spec_attend(*d.values())


def append(L, c=None, **kw):
    d = dict(q=P, qrs=512, qhs=64, k=P, v=P, krs=128, khs=64, vrs=128, vhs=64, dt=sv.BF16, heads=8,
             cache=c or cache(), table=P, slots=10, len=P, ell=None, row=None, rows=20, B=4, gamma=4, turns=P,
             rotary=64, interleaved=0, mscale=1.0, out=P, ws=P, bytes=BIG, stream=None)
    d.update(kw)
    return L.spec_append_kv(*d.values())


def fork(L, c=None, **kw):
    d = dict(table=P, num=P, ref=P, len=P, src=P, dst=P, n=2, B=4, slots=10, cache=c or cache(), status=P, ws=P,
             bytes=BIG, stream=None)
    d.update(kw)
    return L.spec_fork_pages(*d.values())


def compact(L, c=None, **kw):
    d = dict(table=P, num=P, ref=P, B=4, slots=10, cache=c or cache(), out_table=P, out_ref=P, total=P, ws=P, bytes=BIG,
             stream=None)
    d.update(kw)
    return L.spec_compact_pages(*d.values())


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_bad_caches(L, bad, code):
    for call in (attend, append, fork, compact):
        assert call(L, cache(**bad)) == getattr(sv, "ERR_" + code), call.__name__


ALIKE = [(dict(B=-1), "SHAPE"), (dict(B=4097), "SHAPE"), (dict(slots=0), "SHAPE"), (dict(table=None), "NULL"),
         (dict(table=P + 2), "ALIGN"), (dict(ws=None), "NULL"), (dict(ws=P + 8), "ALIGN"), (dict(bytes=16), "WORKSPACE")]
ROWS = ALIKE + [(dict(gamma=-1), "SHAPE"), (dict(gamma=33), "SHAPE"), (dict(rows=19), "SHAPE"), (dict(rows=-1), "SHAPE"),
                (dict(heads=0), "SHAPE"), (dict(dt=sv.E4M3), "SHAPE"), (dict(dt=sv.F16), "SHAPE"),
                (dict(dt=sv.F32), "SHAPE"), (dict(q=None), "NULL"), (dict(out=None), "NULL"), (dict(len=None), "NULL"),
                (dict(q=P + 2), "ALIGN"), (dict(out=P + 8), "ALIGN"), (dict(len=P + 1), "ALIGN"),
                (dict(ell=P + 1), "ALIGN"), (dict(row=P + 1), "ALIGN")]


@pytest.mark.parametrize("bad,code", ROWS + [
    (dict(heads=7), "SHAPE"), (dict(window=-1), "SHAPE"), (dict(sinks=-1), "SHAPE"), (dict(scale=float("nan")), "SHAPE"),
    (dict(scale=float("inf")), "SHAPE"), (dict(rs=4), "ALIGN"), (dict(hs=60), "ALIGN"), (dict(lse=P + 2), "ALIGN")])
def test_attend_refusals(L, bad, code):
    assert attend(L, **bad) == getattr(sv, "ERR_" + code)


@pytest.mark.parametrize("bad,code", ROWS + [
    (dict(rotary=-2), "SHAPE"), (dict(rotary=66), "SHAPE"), (dict(rotary=7), "SHAPE"), (dict(turns=None), "NULL"),
    (dict(turns=P + 4), "ALIGN"), (dict(mscale=float("nan")), "SHAPE"), (dict(mscale=float("inf")), "SHAPE"),
    (dict(k=None), "NULL"), (dict(v=None), "NULL"), (dict(k=P + 8), "ALIGN"), (dict(v=P + 8), "ALIGN"),
    (dict(qrs=1), "ALIGN"), (dict(khs=4), "ALIGN"), (dict(vrs=4), "ALIGN")])
def test_append_refusals(L, bad, code):
    assert append(L, **bad) == getattr(sv, "ERR_" + code)


def test_e4m3_cache_needs_16_bit_rows(L):
    c = cache(dt=sv.E4M3)
    assert attend(L, c, dt=sv.F32) == sv.ERR_SHAPE
    assert append(L, c, dt=sv.F32) == sv.ERR_SHAPE
    assert attend(L, c, bytes=0) == sv.ERR_WORKSPACE      # with 16-bit rows it is the workspace that is too small
    assert append(L, c, bytes=0) == sv.ERR_WORKSPACE


@pytest.mark.parametrize("bad,code", ALIKE + [
    (dict(n=-1), "SHAPE"), (dict(n=5), "SHAPE"), (dict(src=None), "NULL"), (dict(dst=None), "NULL"),
    (dict(status=None), "NULL"), (dict(num=None), "NULL"), (dict(ref=None), "NULL"), (dict(len=None), "NULL"),
    (dict(src=P + 1), "ALIGN"), (dict(num=P + 1), "ALIGN")])
def test_fork_refusals(L, bad, code):
    assert fork(L, **bad) == getattr(sv, "ERR_" + code)


@pytest.mark.parametrize("bad,code", ALIKE + [
    (dict(total=None), "NULL"), (dict(out_table=None), "NULL"), (dict(out_ref=None), "NULL"), (dict(ref=P + 1), "ALIGN"),
    (dict(bytes=256 + 16 * 100), "WORKSPACE")])
def test_compact_refusals(L, bad, code):
    assert compact(L, **bad) == getattr(sv, "ERR_" + code)


def reserve(L, **kw):
    d = dict(table=P, num=P, ref=P, pages=100, len=P, ell=None, B=4, gamma=4, slots=10, page=16, status=P, ws=P,
             bytes=256, stream=None)
    d.update(kw)
    return L.spec_reserve_pages(*d.values())


def commit(L, **kw):
    d = dict(table=P, num=P, ref=P, pages=100, len=P, acc=P, B=4, slots=10, page=16, window=0, sinks=0, out=P, ws=P,
             bytes=256, stream=None)
    d.update(kw)
    return L.spec_commit_pages(*d.values())


def free(L, **kw):
    d = dict(table=P, num=P, ref=P, pages=100, len=P, requests=P, n=3, B=4, slots=10, ws=P, bytes=256, stream=None)
    d.update(kw)
    return L.spec_free_pages(*d.values())


@pytest.mark.parametrize("bad,code", ALIKE + [(dict(pages=0), "SHAPE"), (dict(num=None), "NULL"), (dict(ref=None), "NULL"),
                                              (dict(len=None), "NULL"), (dict(ref=P + 1), "ALIGN")])
def test_page_refusals(L, bad, code):
    for call in (reserve, commit, free):
        assert call(L, **bad) == getattr(sv, "ERR_" + code), call.__name__


def test_page_refusals_of_each(L):
    assert reserve(L, gamma=33) == reserve(L, gamma=-1) == reserve(L, page=0) == sv.ERR_SHAPE
    assert reserve(L, status=None) == sv.ERR_NULL and reserve(L, ell=P + 2) == sv.ERR_ALIGN
    assert commit(L, page=0) == commit(L, window=-1) == commit(L, sinks=-1) == sv.ERR_SHAPE
    assert commit(L, acc=None) == commit(L, out=None) == sv.ERR_NULL
    assert free(L, n=-1) == free(L, n=4097) == sv.ERR_SHAPE
    assert free(L, requests=None) == sv.ERR_NULL and free(L, requests=P + 2) == sv.ERR_ALIGN


def test_nothing_to_do(L):
    assert attend(L, B=0, q=None, out=None, ws=None) == append(L, B=0, q=None, ws=None) == sv.OK
    assert reserve(L, B=0, ws=None) == commit(L, B=0, ws=None) == free(L, n=0, ws=None) == fork(L, n=0, ws=None) == sv.OK


def test_workspace_sizes(L):
    assert L.spec_cache_workspace_bytes(4, 0) >= 256 and L.spec_cache_workspace_bytes(4, 1000) >= 16256
    assert L.spec_cache_workspace_bytes(4097, 0) == L.spec_cache_workspace_bytes(-1, 0) == 0
    assert L.spec_cache_workspace_bytes(4, -1) == 0
    size = L.spec_attend_workspace_bytes
    assert size(4, 4, 8, 2, 64) > 0
    assert size(4097, 4, 8, 2, 64) == size(4, 33, 8, 2, 64) == size(4, 4, 7, 2, 64) == 0
    assert size(4, 4, 8, 0, 64) == size(4, 4, 8, 2, 60) == size(4, 4, 8, 2, 512) == 0


def test_status_strings():
    for code in range(-18, 1):
        assert "unknown" not in sv.status_string(code)


def test_the_binding_refuses_before_the_call():
    """Host tensors, and shapes that do not belong together."""
    q, k = torch.zeros(2, 3, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    K = torch.zeros(9, 16, 2, 64, dtype=torch.bfloat16)
    table, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.attend(q, K, K, table, n)
    with pytest.raises(ValueError, match="CUDA"):
        sv.append_kv(q, k, k, K, K, table, n)
    with pytest.raises(TypeError, match="q must be"):
        sv.attend(q.double(), K, K, table, n)
    with pytest.raises(TypeError, match="k_cache must be"):
        sv.attend(q, K.double(), K.double(), table, n)
    with pytest.raises(TypeError, match="v_cache must be"):
        sv.attend(q, K, K.half(), table, n)
    with pytest.raises(ValueError, match="k_cache must be"):
        sv.attend(q, K[0], K[0], table, n)
    with pytest.raises(ValueError, match="shape and strides"):
        sv.attend(q, K, K[:8], table, n)
    with pytest.raises(ValueError, match="gamma is 7"):
        sv.attend(q, K, K, table, n, gamma=7)
    with pytest.raises(ValueError, match="without a row index"):
        sv.attend(q.flatten(0, 1), K, K, table, n)
    with pytest.raises(ValueError, match="with a row index"):
        sv.attend(q, K, K, table, n, row=n, gamma=2)
    with pytest.raises(ValueError, match="need gamma"):
        sv.attend(q.flatten(0, 1), K, K, table, n, row=n)
    for call in (lambda: sv.reserve_pages(table, n, n, n, gamma=2, page_size=16),
                 lambda: sv.commit_pages(table, n, n, n, n, page_size=16),
                 lambda: sv.free_pages(table, n, n, n, n), lambda: sv.compact_pages(table, n, n, K, K),
                 lambda: sv.fork_pages(table, n, n, n, n, n, K, K)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_row_strides():
    """Which views of rows are taken, and the strides they give."""
    def strides(t, B, gamma, packed=False, heads=2, dim=8):
        # the device check is the only one that needs a GPU
        keep, sv._on_device = sv._on_device, lambda *a: None
        try:
            return sv._row_strides("q", t, t.dtype, heads, dim, B, gamma, packed, 0)
        finally:
            sv._on_device = keep

    x = torch.zeros(3, 5, 6, 16)
    assert strides(x[:, :, 1:3, :8], 3, 4) == (15, 96, 16)
    assert strides(x[:, :1, 1:3, :8], 3, 0) == (3, 480, 16)
    assert strides(x[:1, :, 1:3, :8], 1, 4) == (5, 96, 16)
    assert strides(x[:, 0, 1:3, :8], 3, 0, packed=True) == (3, 480, 16)
    assert strides(x[:1, :1, :1, :8], 1, 0, heads=1) == (1, 8, 8)
    with pytest.raises(ValueError, match="equally spaced"):
        strides(x[:, :4, 1:3, :8], 3, 3)
    with pytest.raises(ValueError, match="adjacent"):
        strides(x[:, :, 1:3, ::2], 3, 4)
    with pytest.raises(ValueError, match="must have shape"):
        strides(x, 3, 4)


def test_rope_frequencies():
    f = sv.rope_frequencies(64, 10000.0)
    assert f.dtype == np.float64 and np.allclose(f, 10000.0 ** (-np.arange(32) / 32), rtol=1e-15)
    assert np.allclose(sv.rope_frequencies(64, scaling="linear", factor=4.0), f / 4, rtol=1e-15)
    b = sv.rope_frequencies(64, scaling="base", factor=8.0)
    assert b[0] == 1.0 and np.isclose(b[-1], f[-1] / 8, rtol=1e-12) and np.all(b[1:] < f[1:])
    n = sv.rope_frequencies(64, scaling="banded", factor=8.0, context=8192)
    waves = 8192 * f / (2 * np.pi)
    assert np.array_equal(n[waves >= 4], f[waves >= 4]) and np.allclose(n[waves <= 1], f[waves <= 1] / 8, rtol=1e-15)
    mid = (waves > 1) & (waves < 4)
    assert mid.any() and np.all(n[mid] < f[mid]) and np.all(n[mid] > f[mid] / 8)
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=-1.0), dict(rotary_dim=8, factor=0.0),
                dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, scaling="banded", factor=2.0),
                dict(rotary_dim=8, scaling="banded", context=10, low=4.0, high=4.0)):
        with pytest.raises(ValueError):
            sv.rope_frequencies(**bad)


def test_rope_table():
    """Fractions of a turn, to 2^-53 of the frequency; negative ones wrap."""
    f = np.array([1.0, 2 * np.pi / 4, 0.0, -2 * np.pi / 4, 1e-6])
    t = sv.rope_table(f, device="cpu")
    got = t.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    assert np.allclose(got, (f / (2 * np.pi)) % 1.0, atol=2.0 ** -50)
    # the product with a far position, wrapped, is the angle of that position
    pos = 1234567
    turn = (t.numpy().view(np.uint64) * np.uint64(pos)).astype(np.float64) / 2.0 ** 64
    d = np.abs(turn - (pos * f / (2 * np.pi)) % 1.0)
    assert np.all(np.minimum(d, 1 - d) < 1e-9)
    with pytest.raises(ValueError):
        sv.rope_table([float("inf")], device="cpu")
