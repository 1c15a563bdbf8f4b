"""Page tables and slot maps of new rows, and the append of rows by their slots,
against plain lists and rotations in 64 bits; a run of them with attention of
shared prefixes."""
import random

import numpy as np
import pytest
import torch

from tests._cache_model import TYPES, Pool, need_pages, rotated
from tests._share_model import Banded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def map_model(pool, new, rows):
    """(status, first, request, position, slot) by the definition of spec_map_rows."""
    free, out = pool.free(), False
    status, first, ends = [], [0], 0
    for b, m in enumerate(new):
        n = pool.len[b]
        ends += max(m, 0)
        first.append(ends)
        need = need_pages(n + m, pool.page) if n >= 0 and m >= 0 else 0
        if m < 0 or n < 0:
            status.append(-16)
        elif m > 0 and ends > rows:
            status.append(-14)
        elif need > pool.slots:
            status.append(-16)
        elif need <= pool.num[b]:
            status.append(0)
        elif out or need - pool.num[b] > len(free):
            out = True
            status.append(-15)
        else:
            for s in range(pool.num[b], need):
                pool.table[b][s] = free.pop(0)
                pool.ref[pool.table[b][s]] = 1
            pool.num[b] = need
            status.append(0)
    request, position, slot = [-1] * rows, [-1] * rows, [-1] * rows
    for b, m in enumerate(new):
        for j in range(max(m, 0)):
            r, p = first[b] + j, pool.len[b] + j
            if r >= rows:
                break
            request[r] = b
            position[r] = p if pool.len[b] >= 0 else -1
            if status[b] == 0 and 0 <= pool.table[b][p // pool.page] < pool.pages:
                slot[r] = pool.table[b][p // pool.page] * pool.page + p % pool.page
    return status, first, request, position, slot


def map_call(sv, pool, new, rows, **kw):
    table, num, ref, length = pool.tensors()
    first, request, position, slot, status, ws = sv.map_rows(table, num, ref, length, i32(new), rows=rows,
                                                             page_size=pool.page, **kw)
    return (table, num, ref, length), (status.tolist(), first.tolist(), request.tolist(), position.tolist(),
                                       slot.tolist()), ws


@pytest.mark.parametrize("B,pages,page,most", [(1, 9, 16, 100), (5, 40, 1, 9), (33, 400, 5, 60), (300, 20000, 16, 900),
                                               (64, 300000, 64, 4000), (4096, 30000, 16, 90)])
def test_random_maps(sv, B, pages, page, most):
    """Steps of prompts and single tokens, pools that run out, ends of requests between them."""
    r = random.Random(B)
    pool = Pool(B, 2 * most // page + 6, pages, page)
    for step in range(4):
        new = [r.choice([0, 1, 1, r.randint(0, most)]) for _ in range(B)]
        rows = max(0, sum(new) + r.choice([0, 7, 0, -new[-1] // 2]))
        want = None
        state, got, ws = map_call(sv, pool, new, rows)
        want = map_model(pool, new, rows)
        assert got == want
        assert sv.read_status(ws) in set(want[0]) | ({0} if not any(want[0]) else set())
        pool.same(*state)
        # the rows are appended: the lengths grow by commit, an accept length of new_len - 1
        accept = [m - 1 if e == 0 else -1 for m, e in zip(new, want[0])]
        sv.commit_pages(*state, i32(accept), page_size=page, workspace=ws)
        pool.commit(accept)
        pool.same(*state)
        pool.end(r.sample(range(B), B // 3))


@pytest.mark.parametrize("new", [[9, 0, 5], [4 * 33, 1, 4 * 700 + 1]])
def test_map_is_undone_by_commit(sv, new):
    """What a step took goes back, a few pages or many of a request; a page that has lost its reference is told."""
    pool = Pool(3, 800, 900, 4)
    state, _, ws = map_call(sv, pool, new, sum(new))
    table, num, ref, length = state
    if max(new) > 1000:
        lost = int(table[2, 500])
        ref[lost] = 0
    sv.commit_pages(*state, i32([-1] * 3), page_size=4, workspace=ws)
    assert sv.read_status(ws) == (sv.ERR_PAGE if max(new) > 1000 else 0)
    pool.same(*state)


def test_map_errors(sv):
    pool = Pool(7, 4, 12, 4)
    pool.len = [-3, 0, 13, 0, 2, 0, 0]
    pool.num = [0, 0, 4, 0, 1, 0, 0]
    pool.table[2] = [0, 1, 2, 3]
    pool.table[4] = [4, -1, -1, -1]
    pool.ref = [1] * 5 + [0] * 7
    new = [2, -1, 4, 1, 3, 20, 3]      # negative length, negative number, too many slots, fine, fine, too many, fine
    rows = 2 + 4 + 1 + 3 + 20 + 2      # the last request's rows end behind the arrays
    state, got, ws = map_call(sv, pool, new, rows)
    want = map_model(pool, new, rows)
    assert want[0] == [-16, -16, -16, 0, 0, -16, -14]
    assert got == want
    assert sv.read_status(ws) in (-16, -14)
    pool.same(*state)
    # a held entry that is no page
    pool.table[3][0] = 99
    pool.num = [min(n, 1) for n in pool.num]
    pool.len = [0, 0, 0, 1, 0, 0, 0]
    state, got, ws = map_call(sv, pool, [0, 0, 0, 1, 0, 0, 0], 2)
    assert got[4] == [-1, -1] and got[3] == [1, -1] and got[2] == [3, -1]
    assert sv.read_status(ws) == sv.ERR_PAGE


def test_map_of_nothing(sv):
    pool = Pool(3, 4, 12, 4)
    state, got, ws = map_call(sv, pool, [0, 0, 0], 0)
    assert got == ([0] * 3, [0] * 4, [], [], []) and sv.read_status(ws) == 0
    state, got, ws = map_call(sv, pool, [0, 0, 0], 5)
    assert got[2:] == ([-1] * 5,) * 3 and sv.read_status(ws) == 0
    pool.same(*state)


def test_sums_beyond_the_arrays(sv):
    """Lengths whose sum passes 31 bits: refused, no wrap."""
    pool = Pool(4, 4, 12, 4)
    state, got, ws = map_call(sv, pool, [3, 0x7fffffff, 0x7fffffff, 2], 5)
    assert got[0] == [0, -14, -14, -14]
    assert got[1][:2] == [0, 3] and all(x > 5 for x in got[1][2:])
    assert got[2] == [0, 0, 0, 1, 1] and got[4][3:] == [-1, -1] and min(got[4][:3]) >= 0
    assert state[1].tolist() == [1, 0, 0, 0]


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,cache,dim,rotary", [("bf16", "bf16", 64, 64), ("fp16", "fp16", 80, 20), ("fp32", "fp32", 64, 32),
                                                    ("bf16", "e4m3", 128, 128), ("fp16", "e4m3", 96, 48), ("bf16", "bf16", 64, 0),
                                                    ("bf16", "bf16", 256, 6), ("fp32", "fp32", 8, 2)])
@pytest.mark.parametrize("rows,queries", [(1, True), (37, True), (37, False)])
def test_append_rows(sv, dtype, cache, dim, rotary, interleaved, rows, queries):
    heads, H, page, pages = 3, 2, 5, 30
    g = torch.Generator().manual_seed(rotary + rows)
    fused = torch.randn(rows, heads + 2 * H, dim, generator=g).to(TYPES[dtype])
    position = torch.tensor([[0, 7, 1000003, 131071, 2 ** 31 - 1, -1][i % 6] for i in range(rows)], dtype=torch.int32)
    slot = torch.randperm(pages * page, generator=g)[:rows]
    slot[5::11] = -1
    K = (torch.randn(pages, page, H, dim, generator=g) * 3).to(TYPES[cache])
    V = (torch.randn(pages, page, H, dim, generator=g) * 3).to(TYPES[cache])
    scales = [torch.rand(H, generator=g) * 0.05 + 0.02 if cache == "e4m3" else None for _ in "kv"]
    freq = sv.rope_frequencies(rotary, 10000.0) if rotary else np.zeros(0)
    ms = 1.25 if rotary else 1.0
    x = fused.cuda()
    Kd, Vd = K.cuda(), V.cuda()
    out = torch.full((rows, heads, dim), 7.0, dtype=TYPES[dtype], device="cuda")
    got, ws = sv.append_rows(x[:, :heads] if queries else None, x[:, heads:heads + H], x[:, heads + H:], Kd, Vd,
                             position.cuda(), slot.cuda(), turns=sv.rope_table(freq) if rotary else None,
                             interleaved=interleaved, mscale=ms, k_scale=None if scales[0] is None else scales[0].cuda(),
                             v_scale=None if scales[1] is None else scales[1].cuda(), out_q=out if queries else None)
    assert sv.read_status(ws) == 0
    assert (got is None) if not queries else got.data_ptr() == out.data_ptr()
    eps, ceps = torch.finfo(TYPES[dtype]).eps, torch.finfo(TYPES[cache]).eps

    def near_enough(have, want, e, mag, least):
        # half a step of the type; the turn in fp32: cos and sin to 2^-21 (the angle's rounding to fp32 half
        # turns, times pi, and sincospi), two products and a sum
        return np.all(np.abs(have - want) <= e / 2 * np.abs(want) * 1.01 + mag * 2.0 ** -20 + least)

    f = fused.float().double().numpy()
    o = out.float().double().cpu().numpy()
    kc, vc = (t.float().double().cpu().numpy().reshape(-1, H, dim) for t in (Kd, Vd))
    touched = np.zeros(pages * page, bool)
    for r in range(rows):
        p, s = int(position[r]), int(slot[r])
        if p < 0:
            assert not queries or (o[r] == 7.0).all()
            continue
        mag = np.abs(f[r]).max() * 2 * ms
        if queries:
            assert near_enough(o[r], rotated(f[r, :heads], p, freq, interleaved, ms), eps, mag, 2.0 ** -25)
        if s < 0:
            continue
        touched[s] = True
        for have, want, scale in ((kc[s], rotated(f[r, heads:heads + H], p, freq, interleaved, ms), scales[0]),
                                  (vc[s], f[r, heads + H:], scales[1])):
            m, least = mag, 2.0 ** -25
            if scale is not None:
                sc = scale.double().numpy()[:, None]
                want, m, least = np.clip(want / sc, -448, 448), mag / float(scale.min()), 2.0 ** -10 * 1.01
            assert near_enough(have, want, ceps, m, least)
    for have, was in ((Kd, K), (Vd, V)):
        raw = (lambda t: t.view(torch.uint8)) if cache == "e4m3" else (lambda t: t)
        a, b = raw(have.cpu()).view(-1, H, dim), raw(was).view(-1, H, dim)
        assert torch.equal(a[~touched], b[~touched])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_many_rows_as_append_kv(sv, cache, interleaved):
    """Rows that take several a block are turned and stored as append_kv does, bit for bit."""
    B, gamma, heads, H, dim, page, slots = 210, 14, 6, 2, 64, 16, 5
    g = torch.Generator().manual_seed(8)
    ell = torch.randint(0, gamma + 1, (B,), generator=g).to(torch.int32)
    lens = torch.randint(0, 3 * page, (B,), generator=g).to(torch.int32)
    table = torch.randperm(B * slots, generator=g).to(torch.int32).view(B, slots)
    n = ell + 1
    row = (torch.cumsum(n, 0) - n).to(torch.int32)
    rows = int(n.sum())
    q, k, v = (torch.randn(rows + 1, h, dim, generator=g).bfloat16().cuda() for h in (heads, H, H))
    scales = [torch.rand(H, generator=g).cuda() + 0.1 for _ in range(2)] if cache == "e4m3" else [None, None]
    kw = dict(turns=sv.rope_table(sv.rope_frequencies(dim)), interleaved=interleaved, k_scale=scales[0], v_scale=scales[1])
    K = torch.zeros(B * slots, page, H, dim, device="cuda").to(TYPES[cache])
    V, K1, V1 = K.clone(), K.clone(), K.clone()
    out, out1 = torch.zeros_like(q), torch.zeros_like(q)
    position, slot = torch.full((rows + 1,), -1, dtype=torch.int32), torch.full((rows + 1,), -1)
    for b in range(B):
        for j in range(int(n[b])):
            p, r = int(lens[b]) + j, int(row[b]) + j
            position[r], slot[r] = p, int(table[b, p // page]) * page + p % page
    sv.append_kv(q, k, v, K, V, table.cuda(), lens.cuda(), ell.cuda(), row.cuda(), gamma=gamma, out_q=out, **kw)
    _, ws = sv.append_rows(q, k, v, K1, V1, position.cuda(), slot.cuda(), out_q=out1, **kw)
    assert sv.read_status(ws) == 0
    raw = (lambda x: x.view(torch.uint8)) if cache == "e4m3" else (lambda x: x)
    assert torch.equal(out, out1) and torch.equal(raw(K), raw(K1)) and torch.equal(raw(V), raw(V1))


def test_slots_behind_the_cache_and_in_place(sv):
    q = torch.randn(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.randn(4, 1, 64, device="cuda", dtype=torch.bfloat16)
    K = torch.zeros(2, 4, 1, 64, device="cuda", dtype=torch.bfloat16)
    V = K.clone()
    slot = torch.tensor([8, 3, 1 << 40, -5], device="cuda")
    out, ws = sv.append_rows(q, k, k, K, V, i32([5, 6, 7, 8]), slot)
    assert sv.read_status(ws) == sv.ERR_PAGE
    assert torch.equal(out, q) and torch.equal(K[0, 3], k[1]) and (K[0, :3] == 0).all() and (K[1] == 0).all()
    turns = sv.rope_table(sv.rope_frequencies(64))
    want, _ = sv.append_rows(q.clone(), k, k, K, V, i32([1, 2, 3, 4]), slot, turns=turns)
    got, _ = sv.append_rows(q, k, k, K, V, i32([1, 2, 3, 4]), slot, turns=turns, out_q=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


def test_layouts_and_a_cache_past_32_bits(sv):
    """Heads outside tokens; a slot whose offset passes 2^32 bytes."""
    k = torch.randn(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    K = torch.zeros(6, 2, 8, 64, device="cuda", dtype=torch.bfloat16).permute(0, 2, 1, 3)
    V = torch.zeros_like(K)
    sv.append_rows(None, k, -k, K, V, i32([0, 1, 2]), torch.tensor([47, 8, 3], device="cuda"))
    assert torch.equal(K[5, 7], k[0]) and torch.equal(V[1, 0], -k[1]) and torch.equal(K[0, 3], k[2])
    assert int((K != 0).any(-1).any(-1).sum()) == 3
    big = torch.zeros(40000, 512, 1, 256, device="cuda", dtype=torch.float8_e4m3fn)    # 5.2 GB
    kk = torch.randn(1, 1, 256, device="cuda", dtype=torch.bfloat16)
    slot = 39999 * 512 + 511
    _, ws = sv.append_rows(None, kk, kk, big, big, i32([9]), torch.tensor([slot], device="cuda"))
    assert sv.read_status(ws) == 0
    assert torch.equal(big.view(-1, 256)[slot], kk[0, 0].to(torch.float8_e4m3fn))


# ------------------------------------------------- prompts, branches and rounds
@pytest.mark.parametrize("captured", [False, True])
def test_prompts_branches_and_rounds(sv, captured):
    """Prompts admitted by map_rows and append_rows, branched by fork_pages, and verification rounds over the
    branches with one plan for two layers, against attention over the history recomputed in 64 bits."""
    B, gamma, layers, heads, H, D, page, pages, slots = 6, 3, 2, 4, 2, 64, 8, 120, 24
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = B * (gamma + 1)

    def rand(*s):
        return torch.randn(*s, device="cuda", generator=g)

    table = torch.full((B, slots), -1, dtype=torch.int32, device="cuda")
    num, ref, length = i32([0] * B), i32([0] * pages), i32([0] * B)
    K, V = (torch.zeros(layers, pages, page, H, D, device="cuda") for _ in "kv")
    ws = sv.alloc_cache_workspace(B, pages)
    freq = sv.rope_frequencies(D)
    turns = sv.rope_table(freq)
    history = [[([], []) for _ in range(layers)] for _ in range(B)]        # turned keys, and values, by position

    def remember(b, layer, pos, k, v):
        hk, hv = history[b][layer]
        del hk[pos:], hv[pos:]
        hk.append(rotated(k.double().cpu().numpy(), pos, freq, False))
        hv.append(v.double().cpu().numpy())

    new = [101, 0, 0, 77, 0, 5]
    total = sum(new)
    first, request, position, slot, status, _ = sv.map_rows(table, num, ref, length, i32(new), rows=total + 3,
                                                            page_size=page, workspace=ws)
    assert status.tolist() == [0] * B
    for layer in range(layers):
        k, v = rand(total + 3, H, D), rand(total + 3, H, D)
        sv.append_rows(None, k, v, K[layer], V[layer], position, slot, turns=turns, workspace=ws)
        for b in range(B):
            for j in range(new[b]):
                remember(b, layer, j, k[first[b] + j], v[first[b] + j])
    sv.commit_pages(table, num, ref, length, i32([n - 1 for n in new]), page_size=page, workspace=ws)
    assert length.tolist() == new
    st, _ = sv.fork_pages(table, num, ref, length, i32([0, 0, 3]), i32([1, 2, 4]), K, V, workspace=ws)
    assert st.tolist() == [0, 0, 0]
    for a, b in ((0, 1), (0, 2), (3, 4)):
        history[b] = [(list(x), list(y)) for x, y in history[a]]

    plan, leader, shared = sv.alloc_share_plan(B, gamma, rows), i32([0] * B), i32([0] * B)
    wa = sv.alloc_attend_shared_workspace(B, gamma, heads, H, D, rows)
    ell, accept = i32([0] * B), i32([0] * B)
    q, k, v = (torch.zeros(layers, rows, n, D, device="cuda") for n in (heads, H, H))
    out = torch.zeros_like(q)

    def step():
        trow, _, _ = sv.pack_rows(ell, gamma)
        sv.reserve_pages(table, num, ref, length, ell, gamma=gamma, page_size=page, workspace=ws)
        sv.share_plan(table, length, ell, trow, gamma=gamma, page_size=page, rows=rows, least=16, out_leader=leader,
                      out_shared=shared, plan=plan)
        for i in range(layers):
            qt, _ = sv.append_kv(q[i], k[i], v[i], K[i], V[i], table, length, ell, trow, gamma=gamma, turns=turns,
                                 workspace=ws)
            sv.attend_shared(qt, K[i], V[i], table, plan, gamma=gamma, out=out[i], workspace=wa)
        sv.commit_pages(table, num, ref, length, accept, page_size=page, workspace=ws)

    graph = None
    if captured:
        accept.fill_(-1)                       # a warm-up round that leaves everything as it was
        kept = [t.clone() for t in (K, V)]
        step()
        torch.cuda.synchronize()
        K.copy_(kept[0])
        V.copy_(kept[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    r = random.Random(4)
    n = list(new)
    n[1], n[2], n[4] = n[0], n[0], n[3]
    for turn in range(5):
        ells = [r.randint(0, gamma) for _ in range(B)]
        accs = [r.randint(0, e) for e in ells]
        ell.copy_(i32(ells))
        accept.copy_(i32(accs))
        for t in (q, k, v):
            t.copy_(rand(*t.shape))
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert sv.read_status(ws) == 0 and sv.read_status(wa) == 0 and sv.read_status(plan) == 0
        assert leader.tolist() == [0, 0, 0, 3, 3, 5]
        assert shared.tolist() == [101 // page] * 3 + [77 // page] * 2 + [0]
        at = 0
        for b in range(B):
            for i in range(layers):
                for j in range(ells[b] + 1):
                    remember(b, i, n[b] + j, k[i, at + j], v[i, at + j])
                hk, hv = (np.stack(x) for x in history[b][i])
                for j in range(ells[b] + 1):
                    p = n[b] + j
                    qq = rotated(q[i, at + j].double().cpu().numpy(), p, freq, False)
                    for h in range(heads):
                        s = hk[:p + 1, h * H // heads] @ qq[h] / np.sqrt(D)
                        w = np.exp(s - s.max())
                        want = w @ hv[:p + 1, h * H // heads] / w.sum()
                        # fp32 rows: scores to (D + 8) 2^-24 of their sums of products (below 40), their weights
                        # to twice that, rotations to 2^-20
                        assert np.abs(out[i, at + j, h].double().cpu().numpy() - want).max() <= 4e-4
            at += ells[b] + 1
            n[b] += accs[b] + 1
            for i in range(layers):
                del history[b][i][0][n[b]:], history[b][i][1][n[b]:]
        assert length.tolist() == n


def test_nothing_is_written_beside_the_buffers(sv):
    band = Banded()
    B, slots, pages, page, rows, H, D = 5, 9, 31, 5, 77, 2, 64
    table, num, ref = band((B, slots), torch.int32, -1), band((B,), torch.int32, 0), band((pages,), torch.int32, 0)
    first, request, position = band((B + 1,), torch.int32), band((rows,), torch.int32), band((rows,), torch.int32)
    slot, status, ws = band((rows,), torch.int64), band((B,), torch.int32), band((256,), torch.uint8, 0)
    sv.map_rows(table, num, ref, i32([0] * B), i32([45, 3, 0, 99, 20]), rows=rows, page_size=page, out_first=first,
                out_request=request, out_position=position, out_slot=slot, out_status=status, workspace=ws)
    assert status.tolist() == [0, 0, 0, -14, -14]
    k = torch.randn(rows, H, D, device="cuda")
    q = torch.randn(rows, 3, D, device="cuda")
    K, V, out = band((pages, page, H, D), torch.float32, 0), band((pages, page, H, D), torch.float32, 0), band(q.shape, q.dtype)
    slot[-1] = pages * page                                    # one behind the cache
    position[-1] = 4
    turns = sv.rope_table(sv.rope_frequencies(D))
    sv.append_rows(q, k, k, K, V, position, slot, turns=turns, out_q=out, workspace=ws)
    assert sv.read_status(ws) in (sv.ERR_ROW_INDEX, sv.ERR_PAGE)
    band.check()
