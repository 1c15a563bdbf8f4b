"""Attention of batches that share prefixes, and its plan, against the formula
in 64 bits and plain lists."""
import random

import pytest
import torch

from tests._share_model import Banded, SharedCase, groups

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


def _run(sv, case):
    plan, leader, shared = case.make_plan(sv)
    assert (leader.tolist(), shared.tolist()) == case.model()
    assert sv.read_status(plan) == 0
    out = torch.full(case.q.shape, 7.0, dtype=case.q.dtype, device="cuda")
    lse = torch.full(case.q.shape[:-1], 7.0, device="cuda")
    _, ws = case.call(sv, plan=plan, out=out, out_lse=lse)
    assert sv.read_status(ws) == 0
    case.check(out, lse)
    want = case.expect()[0]
    assert (out.cpu()[torch.isnan(want)] == 7.0).all()     # rows that no request has are as they were
    assert (lse.cpu()[torch.isnan(want[..., 0])] == 7.0).all()
    return out


TYPES = [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("bf16", "e4m3"), ("fp16", "e4m3")]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("gamma,heads,kv_heads", [(0, 8, 2), (0, 3, 3), (4, 8, 1), (16, 12, 2), (32, 16, 1), (2, 5, 1)])
def test_types_and_groups(sv, dtype, cache, gamma, heads, kv_heads):
    lens = [64, 0, 63, 64, 130, 301, 97]
    ell = [gamma, 0, gamma // 2, gamma, gamma, gamma // 3, gamma]
    _run(sv, SharedCase(share=[([0, 3, 4], 4), ([2, 5, 6], 3)], lens=lens, ell=ell, gamma=gamma, heads=heads,
                        kv_heads=kv_heads, dtype=dtype, cache=cache, seed=1))


@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128, 192, 256])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "e4m3")])
@pytest.mark.parametrize("gamma", [0, 9])
def test_head_sizes(sv, dim, dtype, cache, gamma):
    _run(sv, SharedCase(share=[([0, 1, 3], 5)], lens=[85, 140, 77, 80], ell=[gamma, gamma, gamma // 2, gamma],
                        gamma=gamma, dim=dim, dtype=dtype, cache=cache, heads=8, kv_heads=2, seed=dim))


@pytest.mark.parametrize("page", [1, 3, 5, 16, 24, 64, 100, 128, 256])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("gamma", [0, 16])
def test_page_sizes(sv, page, packed, gamma):
    """Prefixes that end inside a tile, on its border and behind it."""
    pages = max(1, 130 // page)
    n = pages * page
    _run(sv, SharedCase(share=[([0, 2, 3], pages)], lens=[n, 99, n + 128, n + 1], ell=[gamma] * 4, gamma=gamma,
                        page=page, heads=8, kv_heads=2, dim=128, packed=packed, seed=page))


@pytest.mark.parametrize("layout", ["heads", "pair"])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("gamma", [0, 20])
def test_layouts(sv, layout, cache, gamma):
    _run(sv, SharedCase(share=[([0, 1], 4)], lens=[137, 200], ell=[gamma, gamma], gamma=gamma, layout=layout,
                        cache=cache, page=32, dim=128, seed=4))


@pytest.mark.parametrize("dtype,cache,dim,page", [("bf16", "bf16", 128, 64), ("fp16", "e4m3", 64, 16),
                                                  ("bf16", "bf16", 64, 5), ("fp32", "fp32", 64, 16),
                                                  ("bf16", "e4m3", 256, 16)])
@pytest.mark.parametrize("B,gamma", [(40, 8), (150, 0)])
def test_row_tiles_and_split_prefixes(sv, dtype, cache, dim, page, B, gamma):
    """Groups of more rows than a tile, long enough that runs cut the units; packed, ragged."""
    pages = 1300 // page
    r = random.Random(B)
    lens = [pages * page + r.randint(0, 60) for _ in range(B)]
    lens[1] = 3                                                # alone
    case = SharedCase(share=[([b for b in range(B) if b != 1], pages)], lens=lens,
                      ell=[r.randint(0, gamma) for _ in range(B)], gamma=gamma, heads=7, kv_heads=1, dim=dim,
                      dtype=dtype, cache=cache, page=page, packed=True, poison=False, seed=B)
    first = _run(sv, case)
    assert torch.equal(first, _run(sv, case))                  # bit for bit


@pytest.mark.parametrize("gamma", [0, 16])
def test_one_request_and_none_that_share(sv, gamma):
    _run(sv, SharedCase(share=[], lens=[5000], ell=[gamma], gamma=gamma, heads=4, kv_heads=1, dim=64, page=64, seed=1))
    _run(sv, SharedCase(share=[], lens=[0, 16, 700], ell=[0, gamma, gamma], gamma=gamma, heads=4, kv_heads=1, dim=64,
                        seed=2))


def test_rows_at_strides_scale_and_plan_kept(sv):
    """q as a slice of a fused projection, a scale of its own; one plan, two layers."""
    base = dict(share=[([0, 1], 2)], lens=[40, 90], ell=[3, 2], gamma=3, heads=4, kv_heads=2, dim=64)
    one, two = SharedCase(seed=3, **base), SharedCase(seed=3, **base)
    two.k, two.v = two.v, two.k
    plan, _, _ = one.make_plan(sv)
    for case in (one, two):
        wide = torch.full((2, 4, 4 + 2 + 2, 64 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :, 1:5, :64] = case.q.cuda()
        out, ws = case.call(sv, q=wide[:, :, 1:5, :64], plan=plan, scale=-0.2, out=torch.zeros_like(case.q, device="cuda"))
        assert sv.read_status(ws) == 0
        case.check(out, scale=-0.2)


@pytest.mark.parametrize("dtype,cache,dim", [("bf16", "bf16", 128), ("fp16", "e4m3", 64), ("fp32", "fp32", 64),
                                             ("fp16", "fp16", 192)])
def test_invalid_requests_spare_the_others(sv, dtype, cache, dim):
    gamma = 5
    base = dict(share=[([0, 1, 2, 3, 5], 3)], lens=[50, 60, 77, 63, 64, 48], ell=[gamma] * 6, gamma=gamma, heads=8,
                kv_heads=2, dim=dim, page=16, dtype=dtype, cache=cache, seed=5)
    case = SharedCase(**base)
    want = case.expect()
    lens, ell = list(case.lens), list(case.ell)
    lens[1] = case.table.shape[1] * 16 - gamma                 # one position too many
    ell[2] = gamma + 1
    lens[5] = -1
    plan, leader, shared = case.make_plan(sv, lens=lens, ell=ell)
    assert sv.read_status(plan) in (sv.ERR_CACHE_LEN, sv.ERR_VERIFY_LEN)
    seen = [n if b not in (1, 2, 5) else -1 for b, n in enumerate(lens)]
    assert (leader.tolist(), shared.tolist()) == groups(case.table.tolist(), seen, 16, 1)
    out = torch.full(case.q.shape, 7.0, dtype=case.q.dtype, device="cuda")
    _, ws = case.call(sv, plan=plan, out=out)
    assert sv.read_status(ws) in (sv.ERR_CACHE_LEN, sv.ERR_VERIFY_LEN)
    out = out.cpu()
    assert torch.isnan(out[[1, 5]].float()).all() and (out[2] == 7.0).all()
    keep = [0, 3, 4]
    d = (out[keep].double() - want[0][keep]).abs() - want[2][keep]
    assert (d <= 0).all(), float(d.max())


def test_packed_rows_outside_and_behind(sv):
    case = SharedCase(share=[([0, 1, 2], 2)], lens=[40, 33, 50], ell=[2, 1, 0], gamma=4, packed=True, seed=7)
    want = case.expect()
    case.row[1] = 5                                            # rows 5 and 6 of 6
    plan, leader, shared = case.make_plan(sv)
    assert sv.read_status(plan) == sv.ERR_ROW_INDEX
    assert leader.tolist() == [0, 1, 0] and shared.tolist() == [2, 0, 2]
    out = torch.full(case.q.shape, 7.0, dtype=case.q.dtype, device="cuda")
    _, ws = case.call(sv, plan=plan, out=out)
    assert sv.read_status(ws) == sv.ERR_ROW_INDEX
    out = out.cpu().double()
    keep = [0, 1, 2, 5]
    assert ((out[keep] - want[0][keep]).abs() <= want[2][keep]).all()
    assert (out[3:5] == 7.0).all()


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("fp32", 64), ("bf16", 192)])
def test_missing_pages(sv, dtype, dim):
    """A shared page that is missing reaches all of the group, an own one its request."""
    case = SharedCase(share=[([0, 1], 4), ([2, 3], 4)], lens=[70, 80, 70, 90], ell=[2] * 4, gamma=2, dtype=dtype,
                      cache=dtype, dim=dim, seed=9)
    want = case.expect()
    plan, _, _ = case.make_plan(sv)
    table = case.table.clone()
    table[0, 1] = case.k.shape[0]          # the group's pages are its head's
    table[3, 5] = -1
    out, ws = case.call(sv, plan=plan, table=table)
    assert sv.read_status(ws) == sv.ERR_PAGE
    out = out.cpu().double()
    assert torch.isnan(out[[0, 1, 3]]).all()
    assert ((out[2] - want[0][2]).abs() <= want[2][2]).all()


@pytest.mark.parametrize("dtype,heads,gamma", [("bf16", 2, 0), ("bf16", 8, 16), ("fp16", 4, 3), ("fp32", 4, 3)])
def test_values_that_are_not_finite(sv, dtype, heads, gamma):
    """In a shared page they reach all rows of the group; a drafted one the rows that see it."""
    base = dict(share=[([0, 1], 4)], lens=[70, 66, 9], ell=[gamma, gamma, 0], gamma=gamma, heads=heads, kv_heads=1,
                dim=64, dtype=dtype, cache=dtype, seed=8)
    clean, dirty, late = (SharedCase(**base) for _ in range(3))
    page = int(dirty.table[0, 1])
    dirty.v[page, 3, 0, 5] = float("nan")
    dirty.v[page, 3, 0, 7] = float("inf")
    a, b = clean.call(sv)[0].float().cpu(), dirty.call(sv)[0].float().cpu()
    assert torch.equal(a[2, :1], b[2, :1])
    assert torch.isnan(b[:2, :, :, 5]).all() and (~torch.isfinite(b[:2, :, :, 7])).all()
    other = [d for d in range(64) if d not in (5, 7)]
    assert torch.equal(a[:2][..., other], b[:2][..., other])
    if gamma:
        late.v[int(late.table[0, 71 // 16]), 71 % 16, 0, 5] = float("nan")
        late.k[int(late.table[1, 67 // 16]), 67 % 16, 0, 0] = float("nan")
        c = late.call(sv)[0].float().cpu()
        assert torch.equal(a[0, 0], c[0, 0]) and torch.isnan(c[0, 1:, :, 5]).all()
        assert torch.equal(a[0][..., other], c[0][..., other])
        assert torch.equal(a[1, 0], c[1, 0]) and torch.isnan(c[1, 1:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_one_side_far_above_the_other(sv, dtype):
    """The shared positions' scores thousands above the others', and below: no overflow, nothing lost."""
    for sign in (1.0, -1.0):
        case = SharedCase(share=[([0, 1], 2)], lens=[40, 50], ell=[1, 1], gamma=1, heads=2, kv_heads=1, dim=64,
                          dtype=dtype, cache=dtype, seed=6)
        case.q.fill_(1.0)
        for p in case.table[0, :2].tolist():
            case.k[p] = sign * 40.0
        out, ws = case.call(sv)
        assert sv.read_status(ws) == 0
        case.check(out)


def test_a_plan_of_other_sizes_writes_nothing(sv):
    case = SharedCase(share=[([0, 1], 2)], lens=[40, 50], ell=[1, 1], gamma=1, seed=6)
    plan, _, _ = case.make_plan(sv)
    wide = torch.cat([case.table, torch.full((2, 1), -1, dtype=torch.int32)], 1)
    blank = torch.zeros_like(plan)
    for table, p in ((wide, plan), (case.table, blank)):
        out = torch.full(case.q.shape, 7.0, dtype=case.q.dtype, device="cuda")
        _, ws = case.call(sv, plan=p, table=table, out=out)
        assert sv.read_status(ws) == sv.ERR_PLAN
        assert (out == 7.0).all()


def _tree(r, B, page, roots, branches, slots):
    """A page table whose rows share prefixes of prefixes, and lengths."""
    ids = {}
    table, lens = [], []
    deep = [(r.randint(1, slots // 3), [r.randint(0, slots // 3) for _ in range(branches)]) for _ in range(roots)]
    for b in range(B):
        x = r.randrange(roots)
        y = r.randrange(branches)
        names = [(x, i) for i in range(deep[x][0])] + [(x, y, i) for i in range(deep[x][1][y])]
        names += [("own", b, i) for i in range(slots - len(names))]
        cut = r.choice([0, len(names), r.randint(0, len(names))])
        table.append([ids.setdefault(n, len(ids)) if i < cut else -1 for i, n in enumerate(names)])
        lens.append(min(max(0, cut * page - r.randint(0, page)), slots * page - 40))
    return table, lens


@pytest.mark.parametrize("B,roots,branches,slots,least", [(1, 1, 1, 9, 1), (7, 1, 1, 12, 1), (33, 2, 3, 40, 1),
                                                          (64, 1, 40, 700, 64), (300, 5, 4, 90, 100),
                                                          (1500, 60, 3, 50, 1), (4096, 2, 2, 20, 0)])
def test_plans(sv, B, roots, branches, slots, least):
    r = random.Random(B)
    page = 16
    table, lens = _tree(r, B, page, roots, branches, slots)
    t, n = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (table, lens))
    plan, leader, shared = sv.share_plan(t, n, gamma=2, page_size=page, least=least)
    assert sv.read_status(plan) == 0
    want = groups(table, lens, page, least)
    assert leader.tolist() == want[0]
    assert shared.tolist() == want[1]


def test_a_plan_and_its_layers_in_a_graph_while_another_runs(sv):
    """Two captured rounds on two streams, each with its plan and workspace, lengths changing between replays."""
    cases = [SharedCase(share=[([0, 1, 2], 3)], lens=[60, 70, 48], ell=[2, 2, 1], gamma=2, heads=8, kv_heads=2,
                        dim=64, seed=s, poison=False) for s in (1, 2)]
    rounds = []
    for c in cases:
        s = torch.cuda.Stream()
        k, v = c.caches()
        t = dict(k=k, v=v, q=c.q.cuda(), table=c.table.cuda(), n=torch.tensor(c.lens, dtype=torch.int32).cuda(),
                 e=torch.tensor(c.ell, dtype=torch.int32).cuda(), plan=sv.alloc_share_plan(3, 2),
                 leader=torch.zeros(3, dtype=torch.int32).cuda(), shared=torch.zeros(3, dtype=torch.int32).cuda(),
                 ws=sv.alloc_attend_shared_workspace(3, 2, 8, 2, 64), outs=[torch.zeros_like(c.q).cuda() for _ in "ab"])

        def go(t=t):
            sv.share_plan(t["table"], t["n"], t["e"], gamma=2, page_size=16, least=1, out_leader=t["leader"],
                          out_shared=t["shared"], plan=t["plan"])
            for o, (a, b) in zip(t["outs"], ((t["k"], t["v"]), (t["v"], t["k"]))):
                sv.attend_shared(t["q"], a, b, t["table"], t["plan"], out=o, workspace=t["ws"])

        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            go()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            go()
        rounds.append((s, g, t))
    for n in ([60, 70, 48], [48, 49, 62], [20, 77, 62]):
        for c, (s, g, t) in zip(cases, rounds):
            c.lens = n
            t["n"].copy_(torch.tensor(n, dtype=torch.int32))
        torch.cuda.synchronize()
        for s, g, t in rounds:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, (s, g, t) in zip(cases, rounds):
            assert sv.read_status(t["ws"]) == 0 and sv.read_status(t["plan"]) == 0
            assert (t["leader"].tolist(), t["shared"].tolist()) == c.model()
            c.check(t["outs"][0])
            c.k, c.v = c.v, c.k
            c.check(t["outs"][1])
            c.k, c.v = c.v, c.k


def test_a_stream_of_its_own_and_results_as_attend(sv):
    """Made buffers belong to the given stream; the result is attend's within the rounding of 16 bits."""
    case = SharedCase(share=[([0, 1, 2], 4)], lens=[70, 64, 99], ell=[3, 3, 3], gamma=3, heads=8, kv_heads=2, dim=128,
                      seed=4)
    s = torch.cuda.Stream()
    k, v = case.caches()
    q, table = case.q.cuda(), case.table.cuda()
    n, e = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (case.lens, case.ell))
    torch.cuda.synchronize()
    plan, _, _ = sv.share_plan(table, n, e, gamma=3, page_size=16, least=1, stream=s)
    out, ws = sv.attend_shared(q, k, v, table, plan, stream=s)
    assert sv.read_status(ws, s) == 0
    case.check(out)
    ref, _ = sv.attend(q, k, v, table, n, e)
    d = (out.float() - ref.float()).abs()
    assert (d <= 2.0 ** -6 * (1.0 + ref.float().abs())).all()


def test_a_wait_that_runs_out(sv):
    """The tensor-core kernel's timeout path: a status, no fault, and the next call is right again."""
    case = SharedCase(share=[([0, 1], 4)], lens=[300, 400], ell=[8, 8], gamma=8, heads=8, kv_heads=2, dim=128, seed=4)
    sv.selftest_expire_first_wait(True)
    try:
        _, ws = case.call(sv)
        assert sv.read_status(ws) == sv.ERR_TIMEOUT
    finally:
        sv.selftest_expire_first_wait(False)
    _run(sv, case)


def test_empty_batches(sv):
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    table = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    plan, leader, shared = sv.share_plan(table, none, gamma=2, page_size=16)
    assert leader.numel() == shared.numel() == 0
    q = torch.zeros(0, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, ws = sv.attend_shared(q, k, k, table, plan)
    assert out.shape == q.shape and sv.read_status(ws) == 0


def test_rows_behind_the_last_and_a_plan_used_again(sv):
    """Packed rows with room behind them; the same plan for a cache of another type and other heads."""
    base = dict(share=[([0, 1, 2], 3)], lens=[60, 48, 71], ell=[2, 0, 1], gamma=3, dim=64, packed=True, seed=3)
    cases = [SharedCase(heads=8, kv_heads=2, **base), SharedCase(heads=6, kv_heads=6, dtype="fp32", cache="fp32", **base),
             SharedCase(heads=8, kv_heads=1, dtype="fp16", cache="e4m3", **base)]
    for c in cases:
        c.q = torch.cat([c.q, torch.randn(4, *c.q.shape[1:]).to(c.q.dtype)])
    plan, leader, _ = cases[0].make_plan(sv)
    assert leader.tolist() == [0, 0, 0]
    for c in cases:
        out = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda")
        c.table = cases[0].table          # the pages of the plan
        _, ws = c.call(sv, plan=plan, out=out)
        assert sv.read_status(ws) == 0
        c.check(out)
        assert (out[-4:] == 7.0).all()


@pytest.mark.parametrize("dtype,cache,dim", [("bf16", "bf16", 64), ("fp16", "e4m3", 128), ("bf16", "bf16", 192), ("fp32", "fp32", 64)])
def test_many_requests_as_attend(sv, dtype, cache, dim):
    """More items than a block has threads: 1500 requests in 30 groups, and some alone."""
    B, page, H, heads, gamma = 1500, 16, 1, 2, 1
    g = torch.Generator().manual_seed(5)
    r = random.Random(5)
    deep = [r.randint(1, 6) for _ in range(30)]
    pool, table, lens, ell = sum(deep), [], [], []
    start = [sum(deep[:i]) for i in range(30)]
    for b in range(B):
        x = r.randrange(33)
        common = list(range(start[x], start[x] + deep[x])) if x < 30 else []
        n = len(common) * page + r.randint(0, 40)
        own = -(-(n + gamma + 1) // page) - len(common)
        table.append(common + list(range(pool, pool + own)))
        pool += own
        lens.append(n)
        ell.append(r.randint(0, gamma))
    slots = max(map(len, table))
    t = torch.tensor([x + [-1] * (slots - len(x)) for x in table], dtype=torch.int32, device="cuda")
    n, e = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, ell))
    types = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
    k, v = (torch.randn(pool, page, H, dim, generator=g).to(types[cache]).cuda() for _ in "kv")
    q = torch.randn(B, gamma + 1, heads, dim, generator=g).to(types[dtype]).cuda()
    plan, leader, shared = sv.share_plan(t, n, e, gamma=gamma, page_size=page, least=1)
    assert (leader.tolist(), shared.tolist()) == groups(t.tolist(), lens, page, 1)
    outs, lses = [torch.full_like(q, 7.0) for _ in "ab"], [torch.full(q.shape[:-1], 7.0, device="cuda") for _ in "ab"]
    _, ws = sv.attend_shared(q, k, v, t, plan, out=outs[0], out_lse=lses[0])
    _, wa = sv.attend(q, k, v, t, n, e, out=outs[1], out_lse=lses[1])
    assert sv.read_status(ws) == 0 and sv.read_status(wa) == 0
    # both are within the rounding of the output and of the weights of the same sums
    eps = torch.finfo(types[dtype]).eps
    d = (outs[0].double() - outs[1].double()).abs()
    assert (d <= 4 * eps * (1.0 + outs[1].double().abs()) + 2.0 ** -17).all(), float(d.max())
    assert ((lses[0] - lses[1]).abs() <= 2.0 ** -16 * (1.0 + lses[1].abs())).all()


@pytest.mark.parametrize("dtype,cache,dim,page", [("bf16", "bf16", 128, 16), ("fp16", "e4m3", 64, 8), ("fp32", "fp32", 80, 5),
                                                  ("fp16", "fp16", 256, 16)])
def test_nothing_is_written_beside_the_buffers(sv, dtype, cache, dim, page):
    n0 = 48 // page * page
    c = SharedCase(share=[([0, 2, 3], n0 // page)], lens=[n0, 9, n0 + 70, n0 + 1], ell=[4, 0, 3, 4], gamma=4, heads=6,
                   kv_heads=2, dim=dim, dtype=dtype, cache=cache, page=page, packed=True, seed=2)
    c.ell[3] = 9                                              # an error among them
    band = Banded()
    rows = c.q.shape[0]
    L = sv.lib()
    plan = band((L.spec_share_plan_bytes(4, 4, rows),), torch.uint8, 0)
    ws = band((L.spec_attend_shared_workspace_bytes(4, 4, rows, 6, 2, dim),), torch.uint8, 0)
    leader, shared = band((4,), torch.int32), band((4,), torch.int32)
    out, lse = band(c.q.shape, c.q.dtype), band(c.q.shape[:-1], torch.float32)
    c.make_plan(sv, plan=plan, out_leader=leader, out_shared=shared)
    c.call(sv, plan=plan, out=out, out_lse=lse, workspace=ws)
    assert sv.read_status(ws) == sv.ERR_VERIFY_LEN
    band.check()
