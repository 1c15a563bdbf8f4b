"""Slot maps and appends by slot of the sizes whose launches differ: rows by
several words a warp and steps of the whole grid, rows of many values two a block;
and the status word of maps that fail."""
import random

import pytest
import torch

from tests._cache_model import TYPES, Pool
from tests.test_gpu_rows import i32, map_call, map_model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("B,most,rows", [(700, 600, 200_000), (60, 45_000, 1_500_000), (4000, 700, 1_300_000)])
def test_large_maps(sv, B, most, rows):
    """Several words a warp, and (from 1.3 million rows on) several steps of the grid; requests without rows, with few,
    refused ones and rows behind the last."""
    r = random.Random(B)
    page = 64
    pool = Pool(B, most // page + 3, rows // page + 2 * B, page)
    for _ in range(2):
        new = [r.choice([0, 1, r.randint(0, 40), r.randint(0, most)]) for _ in range(B)]
        new[B // 3] = most + 4 * page                 # more slots than the table has
        new[B // 2] = -5
        scale = rows * 0.97 / sum(max(m, 0) for m in new)
        new = [m if m <= 1 or m > most else min(most, int(m * scale)) for m in new]
        state, got, ws = map_call(sv, pool, new, rows)
        want = map_model(pool, new, rows)
        assert -16 in want[0] and -1 in want[2]
        assert got == want
        assert sv.read_status(ws) in {e for e in want[0] if e}
        pool.same(*state)
        accept = [min(m - 1, 20) if e == 0 else -1 for m, e in zip(new, want[0])]  # the rest of a step's pages go back
        sv.commit_pages(*state, i32(accept), page_size=page, workspace=ws)
        pool.commit(accept)
        pool.same(*state)


@pytest.mark.parametrize("new,rows,want", [([9, 40, 1], 50, -15), ([9, 4, 40], 20, -14), ([5, 200, 0], 300, -16),
                                           ([5, 4, 0], 9, 0)])
def test_status_word_of_a_map(sv, new, rows, want):
    """A request that gets no pages, no rows or no slots sets the word, and no other one does."""
    pool = Pool(3, 12, 6, 4)
    state, got, ws = map_call(sv, pool, new, rows)
    model = map_model(pool, new, rows)
    assert got == model and set(model[0]) - {0} == ({want} if want else set())
    assert sv.read_status(ws) == want
    pool.same(*state)


SHAPES = [("bf16", "bf16", 32, 8, 128, 128), ("bf16", "e4m3", 32, 8, 128, 64), ("fp16", "fp16", 9, 9, 96, 12),
          ("fp32", "fp32", 32, 8, 128, 128), ("fp16", "e4m3", 7, 1, 256, 128), ("bf16", "bf16", 8, 8, 80, 0),
          ("fp32", "fp32", 12, 3, 80, 6)]


@pytest.mark.parametrize("dtype,cache,heads,H,dim,rotary", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows", [1311, 1400])
def test_rows_of_many_values(sv, dtype, cache, heads, H, dim, rotary, interleaved, rows):
    """More work items than a block has threads, two rows a block, the last one alone where `rows` is odd: the
    rotation in 64 bits, and append_kv's results bit for bit; out_q may be q."""
    page, slots, gamma = 16, 3, 9
    B = rows // (gamma + 1) + 1
    g = torch.Generator(device="cuda").manual_seed(rows + dim)
    ell = torch.full((B,), gamma, dtype=torch.int32)
    ell[-1] = rows - (B - 1) * (gamma + 1) - 1
    if ell[-1] < 0:
        B, ell = B - 1, ell[:-1]
    lens = torch.tensor([(b * 7) % 30 for b in range(B)], dtype=torch.int32)
    table = torch.randperm(B * slots, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, slots)
    row = torch.arange(B, dtype=torch.int32) * (gamma + 1)
    b = torch.arange(rows) // (gamma + 1)
    position = (lens[b] + torch.arange(rows) % (gamma + 1)).to(torch.int32)
    slot = table[b, position // page].long() * page + position % page
    q, k, v = (torch.randn(rows, h, dim, device="cuda", generator=g).to(TYPES[dtype]) for h in (heads, H, H))
    scales = [torch.rand(H, device="cuda", generator=g) * 0.05 + 0.02 if cache == "e4m3" else None for _ in "kv"]
    freq = sv.rope_frequencies(rotary) if rotary else None
    kw = dict(turns=sv.rope_table(freq) if rotary else None, interleaved=interleaved, mscale=1.25 if rotary else 1.0,
              k_scale=scales[0], v_scale=scales[1])
    K = torch.zeros(B * slots, page, H, dim, device="cuda").to(TYPES[cache])
    V, K1, V1 = K.clone(), K.clone(), K.clone()
    out = torch.empty_like(q)
    sv.append_kv(q, k, v, K, V, table.cuda(), lens.cuda(), ell.cuda(), row.cuda(), gamma=gamma, out_q=out, **kw)
    inplace = q.clone()
    got, ws = sv.append_rows(inplace, k, v, K1, V1, position.cuda(), slot.cuda(), out_q=inplace, **kw)
    assert sv.read_status(ws) == 0 and got.data_ptr() == inplace.data_ptr()

    # half a step of the type; the turn in fp32: cos and sin to 2^-21 (the angle's rounding to fp32 half turns,
    # times pi, and sincospi), two products and a sum
    def turned(x):
        x = x.double()
        if not rotary:
            return x
        a = position.cuda().double()[:, None] * torch.as_tensor(freq, dtype=torch.float64, device="cuda")
        c, s, half = a.cos()[:, None] * 1.25, a.sin()[:, None] * 1.25, rotary // 2
        y = x.clone()
        i, j = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, half), slice(half, rotary))
        y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
        return y

    def near(have, want, t, mag, least):
        d = (have.float().double() - want).abs()
        assert (d <= torch.finfo(TYPES[t]).eps / 2 * want.abs() * 1.01 + mag * 2.0 ** -20 + least).all(), float(d.max())

    mag = max(float(x.float().abs().max()) for x in (q, k, v)) * 2 * 1.25
    near(got, turned(q), dtype, mag, 2.0 ** -25)
    for have, want, scale in ((K1, turned(k), scales[0]), (V1, v.double(), scales[1])):
        m, least = mag, 2.0 ** -25
        if scale is not None:
            want, m, least = (want / scale.double()[:, None]).clamp(-448, 448), mag / 0.02, 2.0 ** -10 * 1.01
        near(have.float().view(-1, H, dim)[slot.cuda()], want, cache, m, least)
    raw = (lambda x: x.view(torch.uint8)) if cache == "e4m3" else (lambda x: x)
    assert torch.equal(out, got) and torch.equal(raw(K), raw(K1)) and torch.equal(raw(V), raw(V1))
