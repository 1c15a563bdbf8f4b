"""Attention over the paged cache against the formula in 64 bits."""
import itertools

import pytest
import torch

from tests._cache_model import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


def _run(sv, case):
    shape = case.q.shape
    out = torch.full(shape, 7.0, dtype=case.q.dtype, device="cuda")
    lse = torch.full(shape[:-1], 7.0, device="cuda")
    _, ws = case.call(sv, out=out, out_lse=lse)
    assert sv.read_status(ws) == 0
    case.check(out, lse)
    # rows that no request has are as they were
    want = case.expect()[0]
    assert (out.cpu()[torch.isnan(want)] == 7.0).all()
    return out


TYPES = [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("bf16", "e4m3"), ("fp16", "e4m3")]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("gamma,heads,kv_heads", [(0, 8, 2), (0, 3, 3), (4, 8, 1), (16, 12, 2), (32, 16, 1), (2, 5, 1)])
def test_types_and_groups(sv, dtype, cache, gamma, heads, kv_heads):
    lens = [0, 1, 63, 64, 130, 301]
    ell = [gamma, 0, gamma // 2, gamma, gamma, gamma // 3]
    _run(sv, Case(lens=lens, ell=ell, gamma=gamma, heads=heads, kv_heads=kv_heads, dtype=dtype, cache=cache, seed=1))


@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128, 192, 256])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "e4m3")])
@pytest.mark.parametrize("gamma", [0, 9])
def test_head_sizes(sv, dim, dtype, cache, gamma):
    _run(sv, Case(lens=[5, 140, 77], ell=[gamma, gamma, gamma // 2], gamma=gamma, dim=dim, dtype=dtype, cache=cache,
                  heads=8, kv_heads=2, seed=dim))


@pytest.mark.parametrize("page", [1, 3, 5, 16, 24, 64, 100, 128, 256])
@pytest.mark.parametrize("gamma", [0, 16])
def test_page_sizes(sv, page, gamma):
    _run(sv, Case(lens=[0, 99, 128, 260], ell=[gamma] * 4, gamma=gamma, page=page, heads=8, kv_heads=2, dim=128,
                  seed=page))


@pytest.mark.parametrize("layout", ["heads", "pair"])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("gamma", [0, 20])
def test_layouts(sv, layout, cache, gamma):
    _run(sv, Case(lens=[37, 200], ell=[gamma, gamma], gamma=gamma, layout=layout, cache=cache, page=32, dim=128,
                  seed=4))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 1), (64, 4), (100, 70), (1000, 4), (63, 64), (64, 200)])
@pytest.mark.parametrize("gamma,cache", [(0, "bf16"), (5, "bf16"), (16, "bf16"), (16, "e4m3")])
def test_windows(sv, window, sinks, gamma, cache, packed):
    lens = [0, 3, 64, 65, 200, 431]
    ell = [gamma, gamma, 0, gamma, gamma // 2, gamma]
    _run(sv, Case(lens=lens, ell=ell, gamma=gamma, window=window, sinks=sinks, packed=packed, page=16, cache=cache,
                  heads=8, kv_heads=2, seed=window))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,kv_heads,longest,gamma", [(1, 1, 5000, 0), (1, 8, 3001, 0), (40, 2, 700, 0),
                                                      (1, 1, 2500, 16), (9, 2, 700, 7)])
def test_long_and_split(sv, dtype, B, kv_heads, longest, gamma):
    lens = [(i * 977 + longest) % (longest + 1) for i in range(B)]
    lens[0] = longest
    case = Case(lens=lens, ell=[gamma] * B, gamma=gamma, heads=4 * kv_heads, kv_heads=kv_heads, dim=64, dtype=dtype,
                cache=dtype, page=64, seed=B)
    first = _run(sv, case)
    assert torch.equal(first, _run(sv, case))      # bit for bit


def test_rows_and_heads_at_strides(sv):
    """q as a slice of a fused projection."""
    case = Case(lens=[20, 90], ell=[3, 2], gamma=3, heads=4, kv_heads=2, dim=64, seed=3)
    wide = torch.full((2, 4, 4 + 2 + 2, 64 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 1:5, :64] = case.q.cuda()
    out, ws = case.call(sv, q=wide[:, :, 1:5, :64], out=torch.zeros_like(case.q, device="cuda"))
    assert sv.read_status(ws) == 0
    case.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gamma,heads", [(4, 2), (16, 8)])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(sv, dtype, gamma, heads):
    base = dict(lens=[70, 9], ell=[gamma, gamma], gamma=gamma, heads=heads, kv_heads=1, dim=64, dtype=dtype, cache=dtype,
                page=16, window=40, sinks=2, seed=8)
    clean, dirty = Case(**base), Case(**base)
    at = 70 + 2                                     # a drafted position: rows 0 and 1 do not see it
    page, off = int(dirty.table[0, at // 16]), at % 16
    dirty.v[page, off, 0, 3] = float("inf")
    dirty.v[page, off, 0, 5] = float("nan")
    old = 70 - 40 + 2                               # rows 0 and 1 alone see this one
    page2, off2 = int(dirty.table[0, old // 16]), old % 16
    dirty.v[page2, off2, 0, 9] = float("-inf")
    a, _ = clean.call(sv)
    b, _ = dirty.call(sv)
    a, b = a.float().cpu(), b.float().cpu()
    assert torch.equal(a[1], b[1])
    for j in range(gamma + 1):
        hit = {3, 5} if j >= 2 else {9}
        for d in range(64):
            if d in hit:
                x = b[0, j, :, d]
                assert (torch.isnan(x) if d == 5 else ~torch.isfinite(x)).all(), (j, d)
            else:
                assert torch.equal(a[0, j, :, d], b[0, j, :, d]), (j, d)


def test_scores_that_are_not_finite(sv):
    """A NaN key at a masked position changes nothing; at a seen one, NaN."""
    base = dict(lens=[40], ell=[3], gamma=3, heads=4, kv_heads=1, dim=64, page=16, seed=2)
    clean, dirty = Case(**base), Case(**base)
    dirty.k[int(dirty.table[0, 42 // 16]), 42 % 16, 0, 0] = float("nan")
    a, b = clean.call(sv)[0].float().cpu(), dirty.call(sv)[0].float().cpu()
    assert torch.equal(a[0, :2], b[0, :2]) and torch.isnan(b[0, 2:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_scores(sv, dtype):
    """One key far above the others, and scores of thousands: no overflow."""
    case = Case(lens=[100, 30], ell=[2, 0], gamma=2, dtype=dtype, cache=dtype, spread=300.0, seed=6)
    out, ws = case.call(sv)
    assert sv.read_status(ws) == 0
    have = ~torch.isnan(case.expect()[0])
    assert torch.isfinite(out.cpu()[have].float()).all()
    case.check(torch.where(have.cuda(), out, torch.zeros_like(out)))


@pytest.mark.parametrize("gamma", [0, 16])
def test_invalid_requests_spare_the_others(sv, gamma):
    case = Case(lens=[50, 20, 77, 33, 64], ell=[gamma] * 5, gamma=gamma, heads=8, kv_heads=2, dim=128, page=16, seed=5)
    good = case.call(sv, out=torch.full(case.q.shape, 7.0, dtype=torch.bfloat16, device="cuda"))[0]
    lens = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
    ell = torch.tensor(case.ell, dtype=torch.int32, device="cuda")
    K, V = case.caches()
    for what, code in (("ell", sv.ERR_VERIFY_LEN), ("long", sv.ERR_CACHE_LEN), ("negative", sv.ERR_CACHE_LEN),
                       ("page", sv.ERR_PAGE), ("pool", sv.ERR_PAGE)):
        l2, e2, t2 = lens.clone(), ell.clone(), case.table.cuda()
        if what == "ell":
            e2[2] = -1
        elif what == "long":
            l2[2] = 16 * t2.shape[1] - gamma
        elif what == "negative":
            l2[2] = -1
        else:
            t2[2, 1] = -1 if what == "page" else K.shape[0]
        out = torch.full(case.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(case.q.shape[:-1], device="cuda")
        _, ws = sv.attend(case.q.cuda(), K, V, t2, l2, e2, out=out, out_lse=lse)
        assert sv.read_status(ws) == code, what
        assert sv.read_status(ws) == 0
        for b in (0, 1, 3, 4):
            # how the work is split may differ, so the last bits may too
            assert torch.allclose(out[b].float(), good[b].float(), rtol=2 ** -6, atol=2 ** -7), (what, b)
        if what == "ell":
            assert (out[2] == 7.0).all()
        else:
            assert torch.isnan(out[2]).all() and torch.isnan(lse[2]).all(), what


def test_packed_rows_out_of_range_are_skipped(sv):
    case = Case(lens=[50, 20, 77], ell=[2, 1, 3], gamma=4, packed=True, seed=5)
    for bad in (-1, case.q.shape[0] - 1, 2 ** 31 - 1):
        row = case.row.clone()
        row[1] = bad
        out = torch.full(case.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        K, V = case.caches()
        _, ws = sv.attend(case.q.cuda(), K, V, case.table.cuda(), torch.tensor(case.lens, dtype=torch.int32).cuda(),
                          torch.tensor(case.ell, dtype=torch.int32).cuda(), row.cuda(), gamma=4, out=out)
        assert sv.read_status(ws) == sv.ERR_ROW_INDEX
        assert (out[3:5] == 7.0).all()
        want = case.expect()
        d = (out.float().double().cpu() - want[0]).abs() - want[2]
        assert (d[:3] <= 0).all() and (d[5:] <= 0).all()


def test_no_verify_lengths_means_gamma(sv):
    case = Case(lens=[30, 3], ell=[6, 6], gamma=6, seed=9)
    K, V = case.caches()
    a, _ = case.call(sv)
    b, _ = sv.attend(case.q.cuda(), K, V, case.table.cuda(), torch.tensor(case.lens, dtype=torch.int32).cuda())
    assert torch.equal(a, b)


def test_scale(sv):
    case = Case(lens=[40], ell=[2], gamma=2, seed=10)
    out, _ = case.call(sv, scale=0.5)
    case.check(out, scale=0.5)
    zero, _ = case.call(sv, scale=0.0)
    case.check(zero, scale=0.0)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("gamma", [0, 16])
def test_negative_scales(sv, dtype, cache, gamma):
    case = Case(lens=[150, 9], ell=[gamma, gamma // 2], gamma=gamma, heads=8, kv_heads=2, dtype=dtype, cache=cache, seed=20)
    if case.k_scale is not None:
        case.k_scale[0] *= -1
        case.v_scale[1] *= -1
    out, ws = case.call(sv, scale=-0.2, out=torch.zeros(case.q.shape, dtype=case.q.dtype, device="cuda"))
    assert sv.read_status(ws) == 0
    case.check(out, scale=-0.2)


@pytest.mark.parametrize("gamma", [0, 16])
def test_on_a_given_stream(sv, gamma):
    """Outputs and workspace made by the call belong to its stream."""
    case = Case(lens=[700, 33], ell=[gamma, gamma], gamma=gamma, heads=8, kv_heads=2, dim=128, seed=21)
    caches, q = case.caches(), case.q.cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                   # the current stream is far behind
    out, ws = case.call(sv, q=q, caches=caches, stream=s)
    s.synchronize()
    with torch.cuda.stream(s):
        got = out.cpu()
    assert sv.read_status(ws, stream=s) == 0
    torch.cuda.synchronize()
    case.check(got)


def test_many_requests(sv):
    """More requests than threads of a block, most of them short."""
    B = 700
    lens = [i % 5 for i in range(B)]
    case = Case(lens=lens, ell=[0] * B, gamma=0, heads=2, kv_heads=1, dim=16, page=4, seed=11)
    _run(sv, case)


@pytest.mark.parametrize("gamma,cache", [(0, "bf16"), (16, "bf16"), (16, "e4m3")])
def test_graph_and_streams(sv, gamma, cache):
    """Captured calls follow the lengths of each replay; calls on two streams
    with their own workspaces do not disturb one another."""
    long = Case(lens=[300, 150], ell=[gamma] * 2, gamma=gamma, dim=128, page=64, cache=cache, seed=12)
    K, V = long.caches()
    q, table = long.q.cuda(), long.table.cuda()
    scales = dict(k_scale=long.to(long.k_scale), v_scale=long.to(long.v_scale))
    lens = torch.tensor(long.lens, dtype=torch.int32, device="cuda")
    out, ws = torch.zeros_like(q), sv.alloc_attend_workspace(2, gamma, 8, 2, 128)
    sv.attend(q, K, V, table, lens, out=out, workspace=ws, **scales)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        for _ in range(3):
            sv.attend(q, K, V, table, lens, out=out, workspace=ws, **scales)
    for new in ([300, 150], [10, 149], [0, 64]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        eager, _ = sv.attend(q, K, V, table, lens, **scales)
        assert torch.equal(out, eager)
    other = torch.cuda.Stream()
    ws2, out2 = sv.alloc_attend_workspace(2, gamma, 8, 2, 128), torch.zeros_like(q)
    torch.cuda.synchronize()
    for _ in range(20):
        sv.attend(q, K, V, table, lens, out=out, workspace=ws, **scales)
        with torch.cuda.stream(other):
            sv.attend(q, K, V, table, lens, out=out2, workspace=ws2, **scales)
    torch.cuda.synchronize()
    assert torch.equal(out, eager) and torch.equal(out2, eager)
    assert sv.read_status(ws) == 0 and sv.read_status(ws2) == 0


def test_offsets_beyond_32_bits(sv):
    """Pages more than 2^31 elements into the cache."""
    pages, page, H, D = 40000, 64, 8, 128          # 2.6e9 elements each
    K = torch.empty(pages, page, H, D, dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    case = Case(lens=[150, 60], ell=[0, 0], gamma=0, heads=8, kv_heads=8, dim=128, page=64, seed=13)
    far = {}
    for b, s in itertools.product(range(2), range(case.table.shape[1])):
        p = int(case.table[b, s])
        if p >= 0:
            far[p] = pages - 1 - p
            K[far[p]] = case.k[p].cuda()
            V[far[p]] = case.v[p].cuda()
    table = torch.tensor([[far.get(int(p), -1) for p in r] for r in case.table], dtype=torch.int32)
    out, ws = sv.attend(case.q.cuda(), K, V, table.cuda(), torch.tensor(case.lens, dtype=torch.int32).cuda())
    assert sv.read_status(ws) == 0
    case.check(out)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 3)])
def test_blocks_with_many_units_of_few_tiles(sv, dim, dtype, cache, window, sinks):
    """Units of one to four tiles, several in a block, of 9 to 85 rows."""
    B, gamma = 170, 16
    lens = [(37 * i) % 131 + 128 * (i % 4) for i in range(B)]
    ell = [(5 * i) % (gamma + 1) for i in range(B)]
    _run(sv, Case(lens=lens, ell=ell, gamma=gamma, heads=10, kv_heads=2, dim=dim, dtype=dtype, cache=cache, page=16,
                  window=window, sinks=sinks, packed=True, seed=31))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("gamma", [4, 16])
def test_e4m3_values_that_are_no_numbers_reach_only_the_rows_that_see_them(sv, dim, gamma):
    base = dict(lens=[130, 9], ell=[gamma, gamma], gamma=gamma, heads=8, kv_heads=1, dim=dim, dtype="bf16", cache="e4m3",
                page=16, window=40, sinks=2, seed=8)
    clean, dirty = Case(**base), Case(**base)
    nan = torch.tensor(float("nan")).to(torch.float8_e4m3fn)

    def put(t, d):
        dirty.v[int(dirty.table[0, t // 16]), t % 16, 0, d] = nan

    put(130 + 2, 3)             # rows 0 and 1 do not see it
    put(130 - 40 + 2, dim - 1)  # rows 0 and 1 alone see it
    put(1, 20)                  # a sink: all rows see it
    a, b = (x.call(sv)[0].float().cpu() for x in (clean, dirty))
    assert torch.equal(a[1], b[1])
    for j in range(gamma + 1):
        hit = {20, 3} if j >= 2 else {20, dim - 1}
        for d in range(dim):
            if d in hit:
                assert torch.isnan(b[0, j, :, d]).all(), (j, d)
            else:
                assert torch.equal(a[0, j, :, d], b[0, j, :, d]), (j, d)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
def test_scale_of_zero_and_masks(sv, cache, dim):
    """All seen keys weigh the same, those that a border hides nothing."""
    case = Case(lens=[300, 0, 126], ell=[16, 9, 3], gamma=16, heads=8, kv_heads=2, dim=dim, cache=cache, window=90, sinks=5,
                seed=12)
    out, ws = case.call(sv, scale=0.0, out=torch.zeros(case.q.shape, dtype=case.q.dtype, device="cuda"))
    assert sv.read_status(ws) == 0
    case.check(out, scale=0.0)
