"""Pages of the cache: reserve, commit, free, fork and compact against plain
lists, the append with rotary positions against 64 bits, and whole rounds."""
import random

import numpy as np
import pytest
import torch

from tests._cache_model import TYPES, Case, Pool, rotated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,pages,page,window,sinks", [(1, 5, 4, 0, 0), (7, 60, 1, 5, 2), (9, 200, 16, 0, 0),
                                                       (40, 700, 3, 20, 7), (16, 600000, 8, 9, 0),
                                                       (1500, 4000, 5, 0, 0)])
def test_random_rounds(sv, B, pages, page, window, sinks):
    """Reserve, commit, fork, free and compact in turn, the pool running out at times."""
    r = random.Random(B)
    gamma, slots = 6, 30
    m = Pool(B, slots, pages, page)
    t, num, ref, lens = m.tensors()
    L = 2
    K = torch.arange(L * pages * page * 8, device="cuda", dtype=torch.float32).view(L, pages, page, 1, 8) \
        if pages <= 4000 else torch.zeros(1, pages, page, 1, 8, device="cuda")
    V = -K
    ws = sv.alloc_cache_workspace(B, pages)
    codes = set()
    for step in range(12):
        ell = [r.randint(0, gamma) for _ in range(B)]
        if step == 3:
            ell[r.randrange(B)] = r.choice([-1, gamma + 1])
        want = m.reserve(ell, gamma)
        got, _ = sv.reserve_pages(t, num, ref, lens, i32(ell), gamma=gamma, page_size=page, workspace=ws)
        assert got.tolist() == want
        codes.update(want)
        m.same(t, num, ref, lens)
        acc = [r.randint(0, ell[b]) if want[b] == 0 else -1 for b in range(B)]
        if step == 5:
            acc[r.randrange(B)] = -1
        m.commit(acc, window, sinks)
        sv.commit_pages(t, num, ref, lens, i32(acc), page_size=page, window=window, sinks=sinks, workspace=ws)
        m.same(t, num, ref, lens)
        if step % 3 == 1 and B > 1:
            ids = list(range(B))
            r.shuffle(ids)
            n = r.randint(1, B // 2)
            dst, src = ids[:n], [r.choice(ids[n:]) for _ in range(n)]
            if step == 7 and n > 2:
                dst[0], dst[1], src[2] = dst[1], dst[1], dst[2]
                dst[2] = B + 3 if B < 20 else dst[2]
            k0, v0 = K.clone(), V.clone()
            want, copies = m.fork(src, dst)
            got, _ = sv.fork_pages(t, num, ref, lens, i32(src), i32(dst), K, V, workspace=ws)
            assert got.tolist() == want
            codes.update(want)
            m.same(t, num, ref, lens)
            for a, b, n in copies:
                k0[:, b, :n], v0[:, b, :n] = k0[:, a, :n], v0[:, a, :n]
            assert torch.equal(K, k0) and torch.equal(V, v0)
        if step % 4 == 3:
            ids = [r.randrange(B) for _ in range(max(1, B // 3))] + [0, 0]
            m.end(ids)
            sv.free_pages(t, num, ref, lens, i32(ids), workspace=ws)
            m.same(t, num, ref, lens)
        if step % 5 == 4:
            k0, v0 = K.clone(), V.clone()
            N, moves = m.compact()
            if step == 4:
                t2, r2 = torch.zeros_like(t), torch.zeros_like(ref)
                total, _ = sv.compact_pages(t, num, ref, K, V, out_page_table=t2, out_ref_count=r2, workspace=ws)
                t.copy_(t2)
                ref.copy_(r2)
            else:
                total, _ = sv.compact_pages(t, num, ref, K, V, workspace=ws)
            assert total.tolist() == [N]
            m.same(t, num, ref, lens)
            if moves:
                a, b = (torch.tensor(x, device="cuda") for x in zip(*moves))
                k0[:, b], v0[:, b] = k0[:, a], v0[:, a]
            assert torch.equal(K, k0) and torch.equal(V, v0)
    if B in (7, 1500):
        assert sv.ERR_POOL in codes


def test_reserve_runs_out_in_order(sv):
    m = Pool(5, 10, 6, 4)
    m.len = [3, 15, 0, 11, 3]           # 1, 4, 1, 3, 1 pages
    t, num, ref, lens = m.tensors()
    st, ws = sv.reserve_pages(t, num, ref, lens, gamma=0, page_size=4)
    assert st.tolist() == m.reserve([0] * 5, 0) == [0, 0, 0, -15, -15]
    m.same(t, num, ref, lens)
    assert sv.read_status(ws) == sv.ERR_POOL


def test_reserve_a_whole_prompt(sv):
    """Slots for a long prompt at once, from a pool of more than one pass of the scan."""
    pages = 700000
    m = Pool(2, 400000, pages, 1)
    m.ref = [1 if i % 3 else 0 for i in range(pages)]
    m.len = [150000, 60000]
    t, num, ref, lens = m.tensors()
    st, _ = sv.reserve_pages(t, num, ref, lens, gamma=3, page_size=1)
    assert st.tolist() == [0, 0]
    free = np.array([i for i in range(pages) if m.ref[i] == 0])
    assert np.array_equal(t[0, :150004].cpu().numpy(), free[:150004])
    assert np.array_equal(t[1, :60004].cpu().numpy(), free[150004:210008])
    assert int((t >= 0).sum()) == 210008 and num.tolist() == [150004, 60004]


def test_errors_of_page_state(sv):
    m = Pool(4, 4, 20, 4)
    m.len = [0, 40, -3, 5]
    t, num, ref, lens = m.tensors()
    st, ws = sv.reserve_pages(t, num, ref, lens, gamma=1, page_size=4)
    assert st.tolist() == [0, -16, -16, 0]
    assert sv.read_status(ws) == sv.ERR_CACHE_LEN
    # a new length beyond the slots, and a bad accept length, leave a request as it was
    before = [x.clone() for x in (t, num, ref, lens)]
    sv.commit_pages(t, num, ref, lens, i32([9, 0, 0, -2]), page_size=4, workspace=ws)
    assert sv.read_status(ws) == sv.ERR_CACHE_LEN
    assert all(torch.equal(a, b) for a, b in zip(before, (t, num, ref, lens)))
    # ids out of range, and a table that names a page twice as often as it is counted
    sv.free_pages(t, num, ref, lens, i32([-1, 4]), workspace=ws)
    assert sv.read_status(ws) == sv.ERR_REQUEST
    assert all(torch.equal(a, b) for a, b in zip(before, (t, num, ref, lens)))
    t[3, 0] = t[0, 0]
    sv.free_pages(t, num, ref, lens, i32([0, 3]), workspace=ws)
    assert sv.read_status(ws) == sv.ERR_PAGE
    assert int(ref.min()) == 0


def test_fork_errors(sv):
    m = Pool(6, 4, 9, 4)
    m.len = [6, 3, 0, 0, 0, 0]
    t, num, ref, lens = m.tensors()
    sv.reserve_pages(t, num, ref, lens, gamma=0, page_size=4)
    m.reserve([0] * 6, 0)
    m.same(t, num, ref, lens)
    K = torch.zeros(9, 4, 2, 8, device="cuda")
    # 7 pages in use and 2 free: one is the first fork's, the second fork's comes
    # from what the destinations give back; then nothing is left
    src, dst = [0, 1, 0, 5, 0], [2, 3, 4, 6, 0]
    want, _ = m.fork(src, dst)
    st, ws = sv.fork_pages(t, num, ref, lens, i32(src), i32(dst), K, K.clone())
    assert st.tolist() == want and want[3] == want[4] == -18
    m.same(t, num, ref, lens)
    assert sv.read_status(ws) == sv.ERR_REQUEST
    # src longer than its slots; its last page missing
    lens[0] = 30
    t[1, 0] = -1
    st, ws = sv.fork_pages(t, num, ref, lens, i32([0, 1]), i32([4, 5]), K, K.clone())
    assert st.tolist() == [-16, -17]


@pytest.mark.parametrize("layout", ["tokens", "heads"])
@pytest.mark.parametrize("cache", ["bf16", "fp32", "e4m3"])
def test_copies_in_layouts(sv, layout, cache):
    """fork and compact on caches with other strides, K and V slices of one array."""
    L, P, page, H, D = 3, 12, 4, 2, 48
    raw = torch.randint(0, 120, (2, L, P, page, H, D), dtype=torch.uint8)
    if layout == "heads":
        mem = raw.permute(0, 1, 2, 4, 3, 5).contiguous().cuda().to(TYPES[cache]).permute(0, 1, 2, 4, 3, 5)
    else:
        mem = raw.cuda().to(TYPES[cache])
    K, V = mem[0], mem[1]
    want = [x.float() for x in (K, V)]
    m = Pool(4, 5, P, page)
    m.len = [7, 11, 0, 0]
    t, num, ref, lens = m.tensors()
    m.reserve([0] * 4, 0)
    sv.reserve_pages(t, num, ref, lens, gamma=0, page_size=page)
    m.end([2, 3])
    sv.free_pages(t, num, ref, lens, i32([2, 3]))
    _, copies = m.fork([1, 0], [2, 3])
    sv.fork_pages(t, num, ref, lens, i32([1, 0]), i32([2, 3]), K, V)
    for x in want:
        for a, b, n in copies:
            x[:, b, :n] = x[:, a, :n]
    m.same(t, num, ref, lens)
    assert all(torch.equal(x.float(), y) for x, y in zip((K, V), want))
    m.end([0])
    sv.free_pages(t, num, ref, lens, i32([0]))
    N, moves = m.compact()
    total, ws = sv.compact_pages(t, num, ref, K, V)
    assert moves and total.tolist() == [N] and sv.read_status(ws) == 0
    for x in want:
        for a, b in moves:
            x[:, b] = x[:, a]
    m.same(t, num, ref, lens)
    assert all(torch.equal(x.float(), y) for x, y in zip((K, V), want))


def test_compact_many_pages(sv):
    """A pool of more than one pass of the scan, in place, and an empty one."""
    P = 600000
    g = torch.Generator(device="cuda").manual_seed(3)
    ref = (torch.rand(P, device="cuda", generator=g) < 0.3).to(torch.int32) * 2
    live = torch.nonzero(ref)[:, 0].to(torch.int32)
    table = live[:2 * 1000].view(2, 1000).clone()
    K = torch.arange(P, device="cuda", dtype=torch.float32).view(P, 1, 1, 1).expand(P, 1, 1, 8).contiguous()
    V = K + 0.5
    N = live.numel()
    holes = torch.nonzero(ref[:N] == 0)[:, 0]
    movers = live[live >= N].long()
    want = torch.arange(P, device="cuda")
    want[movers] = holes
    expect = want[table.long()].to(torch.int32)
    total, ws = sv.compact_pages(table, i32([1000, 900]), ref, K, V)
    assert total.tolist() == [N] and sv.read_status(ws) == 0
    assert torch.equal(table[0], expect[0]) and torch.equal(table[1, :900], expect[1, :900])
    assert (table[1, 900:] == -1).all()
    assert (ref[:N] == 2).all() and (ref[N:] == 0).all()
    assert torch.equal(K[holes, 0, 0, 0].long(), movers) and torch.equal(V[holes, 0, 0, 7], movers + 0.5)
    ref.zero_()
    total, _ = sv.compact_pages(table, i32([0, 0]), ref, K, V)
    assert total.tolist() == [0] and (table == -1).all()


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("bf16", "e4m3"),
                                         ("fp16", "e4m3")])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (64, 0), (80, 20), (96, 24), (128, 64), (128, 2), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_append(sv, dtype, cache, dim, rotary, interleaved, packed):
    gamma, heads, H, page = 3, 4, 2, 8
    lens, ell = [0, 7, 1000003, 131071], [3, 0, 2, 3]
    near = [n % 50 for n in lens]                 # slots needed: the far ones get a shifted table
    c = Case(lens=near, ell=ell, gamma=gamma, heads=heads, kv_heads=H, dim=dim, page=page, dtype=dtype, cache=cache,
             packed=packed, poison=False, seed=rotary)
    slots = max(lens) // page + 2
    table = torch.full((4, slots), -1, dtype=torch.int32)
    for b in range(4):
        for j in range(ell[b] + 1):
            table[b, (lens[b] + j) // page] = c.table[b, (near[b] + j) // page]
    g = torch.Generator().manual_seed(5)
    rows = c.q.shape[:-2]
    k = torch.randn(rows + (H, dim), generator=g).to(c.q.dtype)
    v = torch.randn(rows + (H, dim), generator=g).to(c.q.dtype)
    freq = sv.rope_frequencies(rotary, 10000.0, scaling="linear", factor=3.0) if rotary else np.zeros(0)
    turns = sv.rope_table(freq) if rotary else None
    fused = torch.cat([x for x in (c.q, k, v)], -2).cuda()   # slices of one projection
    K, V = c.caches()
    before = [x.float().cpu().double().numpy() for x in (K, V)]
    out = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda")
    _, ws = sv.append_kv(fused[..., :heads, :], fused[..., heads:heads + H, :], fused[..., heads + H:, :], K, V,
                         table.cuda(), i32(lens), i32(ell), c.to(c.row), gamma=gamma, turns=turns,
                         interleaved=interleaved, mscale=1.25 if rotary else 1.0, k_scale=c.to(c.k_scale),
                         v_scale=c.to(c.v_scale), out_q=out)
    assert sv.read_status(ws) == 0
    got = out.float().cpu().double().numpy().reshape(-1, heads, dim)
    kc, vc = (x.float().cpu().double().numpy() for x in (K, V))
    flat = [x.float().double().numpy().reshape(-1, x.shape[-2], dim) for x in (c.q, k, v)]
    eps = torch.finfo(TYPES[dtype]).eps
    ceps = torch.finfo(TYPES[cache]).eps
    ms = 1.25 if rotary else 1.0
    have = np.zeros(len(got), bool)
    touched = np.zeros(kc.shape[:2], bool)

    def near_enough(x, want, e, mag, least):
        # half a step of the type; the turn in fp32: cos and sin to 2^-21 (the
        # angle's rounding to fp32 half turns, times pi, and sincospi), two
        # products and a sum
        return np.all(np.abs(x - want) <= e / 2 * np.abs(want) * 1.01 + mag * 2.0 ** -20 + least)

    for b in range(4):
        for j in range(ell[b] + 1):
            r, p = c.base(b) + j, lens[b] + j
            have[r] = True
            want = rotated(flat[0][r], p, freq, interleaved, ms)
            assert near_enough(got[r], want, eps, 1.25 * np.abs(flat[0][r]).max(), 2.0 ** -25)
            page_id, off = int(table[b, p // page]), p % page
            touched[page_id, off] = True
            for cachev, x, sc in ((kc, rotated(flat[1][r], p, freq, interleaved, ms), c.k_scale), (vc, flat[2][r], c.v_scale)):
                if sc is not None:
                    x = np.clip(x / sc.double().numpy()[:, None], -448, 448)
                assert near_enough(cachev[page_id, off], x, ceps, 2 * np.abs(x).max(), 2.0 ** -10 if cache == "e4m3" else 2.0 ** -25)
    assert (got[~have] == 7.0).all()
    assert np.array_equal(kc[~touched], before[0][~touched]) and np.array_equal(vc[~touched], before[1][~touched])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_append_a_large_batch(sv, cache, interleaved, packed):
    """Batches that take several rows a block are turned like small ones, bit for bit."""
    B, gamma, heads, H, dim, page = 200, 14, 6, 2, 64, 16
    g = torch.Generator().manual_seed(8)
    ell = torch.randint(-1, gamma + 1, (B,), generator=g).to(torch.int32)
    lens = torch.randint(0, 3 * page, (B,), generator=g).to(torch.int32)
    slots = 5
    table = torch.randperm(B * slots, generator=g).to(torch.int32).view(B, slots).cuda()
    n = (ell + 1).clamp(min=0)
    row = (torch.cumsum(n, 0) - n).to(torch.int32).cuda() if packed else None
    rows = (int(n.sum()),) if packed else (B, gamma + 1)
    q, k, v = (torch.randn(rows + (h, dim), generator=g).bfloat16().cuda() for h in (heads, H, H))
    scales = [torch.rand(H, generator=g).cuda() + 0.1 for _ in range(2)] if cache == "e4m3" else [None, None]
    turns = sv.rope_table(sv.rope_frequencies(dim))
    kw = dict(gamma=gamma, turns=turns, interleaved=interleaved, k_scale=scales[0], v_scale=scales[1])
    K = torch.zeros(B * slots, page, H, dim, device="cuda").to(TYPES[cache])
    V, K1, V1 = K.clone(), K.clone(), K.clone()
    out, out1 = torch.zeros_like(q), torch.zeros_like(q)
    ell, lens = ell.cuda(), lens.cuda()
    _, ws = sv.append_kv(q, k, v, K, V, table, lens, ell, row, out_q=out, **kw)
    assert sv.read_status(ws) == sv.ERR_VERIFY_LEN
    for b in range(0, B, 20):
        s = slice(b, b + 20)
        at = (slice(None),) if packed else (s,)
        sv.append_kv(q[at], k[at], v[at], K1, V1, table[s].contiguous(), lens[s].contiguous(), ell[s].contiguous(),
                     None if row is None else row[s].contiguous(), out_q=out1[at], **kw)
    raw = (lambda x: x.view(torch.uint8)) if cache == "e4m3" else (lambda x: x)
    assert torch.equal(out, out1) and torch.equal(raw(K), raw(K1)) and torch.equal(raw(V), raw(V1))
    assert float(out.float().abs().sum()) > 0 and float(K.float().abs().sum()) > 0


def test_append_in_place_and_clamped(sv):
    """out_q = q; values beyond the 8-bit range are clamped."""
    q = torch.randn(1, 2, 2, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.full((1, 2, 1, 64), 3.0e4, device="cuda", dtype=torch.bfloat16)
    K = torch.zeros(2, 4, 1, 64, device="cuda").to(torch.float8_e4m3fn)
    V = K.clone()
    turns = sv.rope_table(sv.rope_frequencies(64))
    args = (k, -k, K, V, i32([[1]]), i32([2]))
    want, _ = sv.append_kv(q.clone(), *args, turns=turns)
    got, _ = sv.append_kv(q, *args, turns=turns, out_q=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)
    assert (V.float()[1, 2:] == -448).all() and (V.float()[1, :2] == 0).all() and (V.float()[0] == 0).all()


def test_append_without_a_page(sv):
    q = torch.randn(3, 1, 2, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.randn(3, 1, 1, 64, device="cuda", dtype=torch.bfloat16)
    K = torch.zeros(2, 4, 1, 64, device="cuda", dtype=torch.bfloat16)
    V = K.clone()
    for lens, table, code in (([5, 0, 0], [[0, -1], [1, -1], [-1, -1]], sv.ERR_PAGE),
                              ([8, 0, 2], [[0, 0], [1, 1], [2, 0]], sv.ERR_CACHE_LEN),
                              ([-1, 0, 0], [[0, 0], [1, 1], [-5, 0]], sv.ERR_CACHE_LEN)):
        K.zero_()
        V.zero_()
        out, ws = sv.append_kv(q, k, k, K, V, i32(table), i32(lens))
        assert sv.read_status(ws) in (code, sv.ERR_PAGE)
        assert torch.equal(out, q)
        assert torch.equal(K[1, 0], k[1, 0]) and (K[0] == 0).all() and (K[1, 1:] == 0).all()


# --------------------------------------------------------------- whole rounds
def test_rounds_in_a_graph(sv):
    """Schedule, pack, reserve, append, attend, verify and commit in one graph,
    replayed round after round, against the same calls run one by one and
    against attention recomputed over the whole history."""
    B, gamma, V, H, heads, D, page, pages = 6, 4, 500, 2, 4, 64, 8, 80
    g = torch.Generator(device="cuda").manual_seed(2)

    def rand(*s):
        return torch.randn(*s, device="cuda", generator=g)

    embed, head = rand(V, D), rand(D * heads, V) * 0.2
    wq, wk, wv = rand(D, heads * D) * 0.1, rand(D, H * D) * 0.1, rand(D, H * D) * 0.1
    turns = sv.rope_table(sv.rope_frequencies(D))
    rows = B * (gamma + 1)

    class State:
        def __init__(self):
            self.table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
            self.num, self.ref = i32([0] * B), i32([0] * pages)
            self.len = i32([0] * B)
            self.K = torch.zeros(pages, page, H, D, device="cuda")
            self.V = torch.zeros_like(self.K)
            self.conf = torch.zeros(B, gamma, device="cuda")
            self.last = i32([1] * B)
            self.draft = torch.zeros(B, gamma, dtype=torch.int32, device="cuda")
            self.u = torch.zeros(B, gamma + 2, device="cuda")
            self.dlogits = torch.zeros(rows, V, device="cuda")
            self.ws = sv.alloc_cache_workspace(B, pages)
            self.wa = sv.alloc_attend_workspace(B, gamma, heads, H, D)
            self.wv = sv.alloc_verify_workspace(B, gamma, V, sv.F32)
            self.wsched = torch.zeros(256, dtype=torch.uint8, device="cuda")
            self.out = torch.zeros(rows, heads, D, device="cuda")
            self.tok = torch.zeros(B, gamma + 1, dtype=torch.int32, device="cuda")
            self.acc = torch.zeros(B, dtype=torch.int32, device="cuda")
            self.rowtok = torch.zeros(rows, dtype=torch.int64, device="cuda")

        def round(self):
            self.ell, _ = sv.schedule_static(self.conf, 0.5, gamma, 0, workspace=self.wsched)
            trow, drow, _ = sv.pack_rows(self.ell, gamma)
            sv.reserve_pages(self.table, self.num, self.ref, self.len, self.ell, gamma=gamma, page_size=page,
                             workspace=self.ws)
            j = torch.arange(gamma + 1, device="cuda")
            cand = torch.cat([self.last[:, None], self.draft], 1).long()
            at = torch.where(j[None, :] <= self.ell[:, None], trow[:, None].long() + j, rows)
            ext = torch.zeros(rows + 1, dtype=torch.int64, device="cuda")
            ext.scatter_(0, at.view(-1), cand.view(-1))
            self.rowtok.copy_(ext[:rows])
            x = embed[self.rowtok]
            q, k, v = ((x @ w).view(rows, -1, D) for w in (wq, wk, wv))
            q, _ = sv.append_kv(q, k, v, self.K, self.V, self.table, self.len, self.ell, trow, gamma=gamma,
                                turns=turns, workspace=self.ws)
            sv.attend(q, self.K, self.V, self.table, self.len, self.ell, trow, gamma=gamma, out=self.out,
                      workspace=self.wa)
            logits = self.out.reshape(rows, -1) @ head
            sv.verify_packed(logits, self.dlogits, trow, drow, self.draft, self.ell, 1.0, self.u,
                             out_tokens=self.tok, out_accept_len=self.acc, workspace=self.wv)
            sv.commit_pages(self.table, self.num, self.ref, self.len, self.acc, page_size=page, workspace=self.ws)

    a, b = State(), State()
    a.round()                                    # warm-up (modules loaded, workspaces of torch's products)
    a = State()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.round()
    history = [[] for _ in range(B)]
    last = [1] * B
    for step in range(8):
        conf, draft = torch.rand(B, gamma, device="cuda", generator=g), torch.randint(0, V, (B, gamma), device="cuda", generator=g, dtype=torch.int32)
        u = torch.rand(B, gamma + 2, device="cuda", generator=g) * 0.9
        for s in (a, b):
            s.conf.copy_(conf)
            s.draft.copy_(draft)
            s.u.copy_(u)
            s.last.copy_(i32(last))
        graph.replay()
        b.round()
        torch.cuda.synchronize()
        for s in (a, b):
            assert [sv.read_status(w) for w in (s.ws, s.wa, s.wv)] == [0, 0, 0]
        for n in ("table", "num", "ref", "len", "tok", "acc", "K", "V", "ell"):
            assert torch.equal(getattr(a, n), getattr(b, n)), (step, n)
        acc, tok = b.acc.tolist(), b.tok.tolist()
        for i in range(B):
            assert acc[i] >= 0
            history[i] += [last[i]] + tok[i][:acc[i]]
            last[i] = tok[i][acc[i]]
            assert b.len[i] == len(history[i])
    # the cache holds exactly the accepted history, rotated
    freq = sv.rope_frequencies(D)
    for i in range(B):
        x = embed[torch.tensor(history[i], device="cuda")]
        k = (x @ wk).view(-1, H, D).double().cpu().numpy()
        for p in range(len(history[i])):
            got = b.K[int(b.table[i, p // page]), p % page].double().cpu().numpy()
            want = rotated(k[p], p, freq, False)
            assert np.abs(got - want).max() <= 1e-4 * max(1.0, np.abs(want).max())
    assert int(b.ref.sum()) == sum(-(-len(h) // page) for h in history)
