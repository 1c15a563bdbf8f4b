"""Cases that measure attention of a batch that shares long prefixes (with the
plan that finds them), the page tables and slot maps of new rows, and the append
of rows by their slots.

``own`` false: elementary torch operations.  ``own`` true: the package's calls.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
PASSES = 32  # of the plan
LEAST = 256  # positions: shorter prefixes are not shared


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # four samples of one prompt, one new token each: the latency of a decoding step of four layers
        dict(name="shared_samples_small", op="shared", layers=4, B=4, roots=1, branches=1, root=600, branch=0, gamma=0,
             heads=32, kv_heads=8, dim=128, page=16, shortest=1, longest=200, dtype="bf16", cache="bf16", packed=False,
             full=True),
        # one new token for each of 64 chats behind a long system prompt: the chats' own positions bound it
        dict(name="shared_chats_one_token", op="shared", layers=2, B=64, roots=1, branches=1, root=8192, branch=0,
             gamma=0, heads=32, kv_heads=8, dim=128, page=64, shortest=1, longest=2000, dtype="bf16", cache="bf16",
             packed=False, full=True),
        # drafts of 48 questions to three long documents, in packed rows
        dict(name="shared_documents", op="shared", layers=1, B=48, roots=3, branches=1, root=32768, branch=0, gamma=4,
             heads=32, kv_heads=8, dim=128, page=64, shortest=1, longest=500, dtype="bf16", cache="bf16", packed=True,
             full=True),
        # blocks of 16 drafts verified at once (the block-diffusion workload's batch and block) behind one prompt
        dict(name="shared_verify_block", op="shared", layers=1, B=64, roots=1, branches=1, root=8192, branch=0,
             gamma=16, heads=32, kv_heads=8, dim=128, page=64, shortest=500, longest=1500, dtype="bf16", cache="bf16",
             packed=False, full=True),
        # scheduled ragged lengths, a tree of prompts, an 8-bit cache, an odd group of heads
        dict(name="shared_tree_e4m3", op="shared", layers=1, B=64, roots=2, branches=3, root=1000, branch=6000,
             gamma=16, heads=28, kv_heads=4, dim=64, page=16, shortest=1, longest=1500, dtype="fp16", cache="e4m3",
             packed=True, full=False),
        # 32-bit rows of a small model, pages that are no power of two
        dict(name="shared_fp32", op="shared", layers=1, B=12, roots=2, branches=1, root=2000, branch=0, gamma=4,
             heads=8, kv_heads=2, dim=64, page=5, shortest=1, longest=300, dtype="fp32", cache="fp32", packed=False,
             full=False),
        # the plan alone: a chat batch; and a tree of prompts over many requests
        dict(name="plan_small", op="plan", B=16, roots=2, branches=2, root=500, branch=1500, page=16, gamma=4,
             shortest=1, longest=1000),
        dict(name="plan_large", op="plan", B=1024, roots=24, branches=4, root=2000, branch=6000, page=16, gamma=16,
             shortest=1, longest=2000),
        # a step's new rows: a few prompts among single tokens; and a large admission of prompts
        dict(name="map_small", op="map", B=16, page=16, shortest=1, longest=2000, new=100, spare=300, single=0.7),
        dict(name="map_large", op="map", B=256, page=16, shortest=1, longest=300, new=8000, spare=90000, single=0.0),
        # one short prompt's keys and values; and many prompts' at once, into an 8-bit cache
        dict(name="rows_small", op="rows", B=1, heads=32, kv_heads=8, dim=128, rotary=128, page=16, new=100,
             shortest=1, longest=2000, dtype="bf16", cache="bf16", interleaved=False, queries=True),
        dict(name="rows_large", op="rows", B=24, heads=32, kv_heads=8, dim=128, rotary=64, page=32, new=2000,
             shortest=1, longest=1000, dtype="bf16", cache="e4m3", interleaved=True, queries=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "shared", "plan", "map", "rows", "rows"])
    page = rng.choice([1, 5, 8, 16, 16, 32, 48, 64, 64, 128, 256])
    if op == "shared":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp16", "fp32"])
        gamma = rng.choice([0, 0, 1, 3, 4, 7, 8, 13, 16, 32])
        kv_heads = rng.choice([1, 2, 4, 5, 8])
        group = rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
        dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
        B = _log(rng, 2, 96)
        roots, branches = rng.randint(1, max(1, min(6, B // 4))), rng.choice([1, 1, 2, 3])
        cache = dtype if dtype == "fp32" else rng.choice([dtype, dtype, "e4m3"])
        # bounded so that no drawn case has more keys, or more work, than the largest listed ones
        keys = 200_000_000 // (2 * kv_heads * dim * SIZE[cache])
        both = min(keys // (roots * (1 + branches)), 1_500_000_000 // (B * kv_heads * dim),
                   (4_000_000_000 if dtype == "fp32" else 25_000_000_000) // (B * kv_heads * group * (gamma + 1) * dim))
        root = _log(rng, min(300, both), min(40000, both))
        branch = _log(rng, 16, max(16, both - root)) if branches > 1 else 0
        return dict(op=op, layers=rng.choice([1, 1, 2]), B=B, roots=roots, branches=branches, root=root, branch=branch,
                    gamma=gamma, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page, shortest=1,
                    longest=_log(rng, 1, max(2, min(2000, both // 4, keys // B))), dtype=dtype, cache=cache,
                    packed=rng.random() < 0.5, full=rng.random() < 0.5)
    if op == "plan":
        branches = rng.choice([2, 2, 3, 5])
        return dict(op=op, B=_log(rng, 10, 1024), roots=_log(rng, 2, 24), branches=branches, root=_log(rng, 700, 2000),
                    branch=_log(rng, 1, 6000), page=min(max(page, 8), 64), gamma=rng.choice([0, 1, 4, 8, 16, 32]),
                    shortest=1, longest=_log(rng, 1, 2000))
    if op == "map":
        B = _log(rng, 1, 1024)
        new = _log(rng, 1, max(1, min(8000, 1_000_000 // B)))
        return dict(op=op, B=B, page=max(page, 5), shortest=1, longest=_log(rng, 1, 3000), new=new,
                    spare=_log(rng, max(40, B * new // max(page, 5) // 2), 2 * B + B * new // max(page, 5) + 100),
                    single=rng.choice([0.0, 0.3, 0.9]))
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
    group = rng.choice([1, 2, 4, 7])
    B = _log(rng, 1, 64)
    new = _log(rng, 1, max(1, min(4000, 12_000 * 48 * 128 // (B * kv_heads * (group + 2) * dim))))
    return dict(op=op, B=B, heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                rotary=rng.choice([0, dim, dim, dim // 2, dim // 4]), page=page, new=new, shortest=1,
                longest=max(1, min(_log(rng, 1, 100000), 60_000_000 // (B * kv_heads * dim))), dtype=dtype,
                cache=dtype if dtype == "fp32" else rng.choice([dtype, dtype, "e4m3"]),
                interleaved=rng.random() < 0.5, queries=rng.random() < 0.8)


# ------------------------------------------------------- lengths (by the case)
def _pages(n, page):
    return -(-n // page)


def _rng(case, seed=0):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")) + str(seed))


def _tree(case, seed=0):
    """Each request's pages by name, its length and drafts.  For attention they
    belong to the case, so that every seed has the same work; the plan's inputs are
    nothing else, and are of the seed.  A name is ("root", r, i), ("branch", r, s,
    i) or ("own", b, i)."""
    r = _rng(case, seed if case["op"] == "plan" else 0)
    page = case["page"]
    roots = [max(1, r.randint(case["root"] // 2, case["root"]) // page) for _ in range(case["roots"])]
    roots[0] = max(1, case["root"] // page)
    twigs = [[r.randint(case["branch"] // 2, case["branch"]) // page for _ in range(case["branches"])]
             for _ in roots]
    names, lens, ell = [], [], []
    for b in range(case["B"]):
        x = r.randrange(len(roots))
        y = r.randrange(case["branches"])
        common = [("root", x, i) for i in range(roots[x])] + [("branch", x, y, i) for i in range(twigs[x][y])]
        n = len(common) * page + r.randint(case["shortest"], max(case["shortest"], case["longest"]))
        e = case["gamma"] if case.get("full", True) else r.randint(0, case["gamma"])
        names.append(common + [("own", b, i) for i in range(_pages(n + e + 1, page) - len(common))])
        lens.append(n)
        ell.append(e)
    return names, lens, ell


def _grown(case):
    """Cache lengths, and numbers of new rows, of the requests."""
    r = _rng(case)
    lens = [r.randint(case["shortest"], max(case["shortest"], case["longest"])) for _ in range(case["B"])]
    new = [1 if r.random() < case.get("single", 0.0) else r.randint(0 if case["op"] == "map" else 1, case["new"])
           for _ in range(case["B"])]
    new[r.randrange(case["B"])] = case["new"]
    return lens, new


def work(case):
    op = case["op"]
    if op in ("shared", "plan"):
        names, lens, ell = _tree(case)
        entries = sum(len(x) for x in names)
        if op == "plan":
            return dict(bytes=4 * entries + 4 * 5 * case["B"], flops=0)
        keys = {}  # positions of each page that somebody sees
        for x, n, e in zip(names, lens, ell):
            for i, name in enumerate(x):
                keys[name] = max(keys.get(name, 0), min(case["page"], n + e + 1 - i * case["page"]))
        rows = sum(e + 1 for e in ell)
        pairs = sum((e + 1) * (n + 1) + e * (e + 1) // 2 for n, e in zip(lens, ell))
        each = sum(keys.values()) * 2 * case["kv_heads"] * case["dim"] * SIZE[case["cache"]] + \
            2 * rows * case["heads"] * case["dim"] * SIZE[case["dtype"]]
        return dict(bytes=case["layers"] * each + 4 * entries,
                    flops=case["layers"] * 4 * case["dim"] * case["heads"] * pairs)
    lens, new = _grown(case)
    rows = sum(new)
    if op == "map":
        held = sum(_pages(n, case["page"]) for n in lens)
        return dict(bytes=4 * (held + case["spare"]) + 16 * rows + 20 * case["B"], flops=0)
    es, cs = SIZE[case["dtype"]], SIZE[case["cache"]]
    heads = case["heads"] if case["queries"] else 0
    return dict(bytes=rows * (case["dim"] * (2 * heads * es + 2 * case["kv_heads"] * (es + cs)) + 12),
                flops=3 * rows * case["rotary"] * (heads + case["kv_heads"]))


# ---------------------------------------------------------------- the inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _normal(shape, dtype, g, std=1.0):
    """Normal values of `dtype`, made in slices so that the 32-bit ones stay small."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = (torch.randn(n, device="cuda", generator=g) * std).to(dtype)
    return out


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _package():
    import speculative_decoding_verification_softmax_gb300 as sv
    return sv


def _frequencies(case):
    half = case["rotary"] // 2
    return 10000.0 ** (-np.arange(half, dtype=np.float64) / max(half, 1))


def _scales(case, g):
    if case["cache"] != "e4m3":
        return None, None
    return tuple(torch.rand(case["kv_heads"], device="cuda", generator=g) * 0.05 + 0.02 for _ in range(2))


def prepare(case, seed):
    g = _gen(seed, 1)
    op, B, page = case["op"], case["B"], case["page"]
    s = dict(case=case)
    if op in ("shared", "plan"):
        names, lens, ell = _tree(case, seed)
        ids = {}
        rows = [[ids.setdefault(x, len(ids)) for x in r] for r in names]
        pool = len(ids) + 3
        perm = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
        slots = max(len(r) for r in rows)
        named = torch.tensor([r + [-1] * (slots - len(r)) for r in rows], device="cuda")
        s.update(table=torch.where(named >= 0, perm[named.clamp(min=0)], -1).to(torch.int32).contiguous(),
                 cache_len=_ints(lens), verify_len=None if case.get("full", True) else _ints(ell), row=None,
                 leader=torch.zeros(B, dtype=torch.int32, device="cuda"),
                 shared=torch.zeros(B, dtype=torch.int32, device="cuda"))
        total = B * (case["gamma"] + 1)
        if op == "shared":
            L, H, D = case["layers"], case["kv_heads"], case["dim"]
            dt, ct = TYPES[case["dtype"]], TYPES[case["cache"]]
            std = 20.0 if case["cache"] == "e4m3" else 1.0  # entries as a quantised cache holds them
            s.update(k_cache=_normal((L, pool, page, H, D), ct, g, std),
                     v_cache=_normal((L, pool, page, H, D), ct, g, std))
            s["k_scale"], s["v_scale"] = _scales(case, g)
            shape = (B, case["gamma"] + 1)
            if case["packed"]:
                n = np.array([e + 1 for e in ell])
                s["row"] = _ints((np.cumsum(n) - n).tolist())
                total = int(n.sum())
                shape = (total,)
            s["q"] = _normal((L,) + shape + (case["heads"], D), dt, g, 2.0)
            s["out"] = torch.zeros_like(s["q"])
        s["rows"] = total
        if own:
            sv = _package()
            s["plan"] = sv.alloc_share_plan(B, case["gamma"], total)
            if op == "shared":
                s["ws"] = sv.alloc_attend_shared_workspace(B, case["gamma"], case["heads"], H, D, total)
        return s
    lens, new = _grown(case)
    if op == "map":
        held = [_pages(n, page) for n in lens]
        slots = max(_pages(n + m, page) for n, m in zip(lens, new))
        pool = sum(held) + case["spare"]
        taken = torch.randperm(pool, device="cuda", generator=g)[:sum(held)].to(torch.int32)
        start = torch.cumsum(_ints(held), 0) - _ints(held)
        at = torch.arange(slots, device="cuda")[None, :]
        table = torch.where(at < _ints(held)[:, None], taken[(start[:, None] + at).clamp(max=sum(held) - 1)], -1)
        ref = torch.zeros(pool, dtype=torch.int32, device="cuda")
        ref[taken.long()] = 1
        rows = sum(new)
        s.update(table=table.to(torch.int32).contiguous(), num=_ints(held), ref=ref, cache_len=_ints(lens),
                 new_len=_ints(new), none=_ints([-1] * B), rows=rows, first=_ints([0] * (B + 1)),
                 status=_ints([0] * B), request=_ints([0] * rows), position=_ints([0] * rows),
                 slot=torch.zeros(rows, dtype=torch.int64, device="cuda"))
        if own:
            s["ws"] = _package().alloc_cache_workspace(B)
        return s
    H, D = case["kv_heads"], case["dim"]
    dt, ct = TYPES[case["dtype"]], TYPES[case["cache"]]
    held = np.array([_pages(n + m, page) for n, m in zip(lens, new)])
    pool = int(held.sum()) + 3
    perm = torch.randperm(pool, device="cuda", generator=g)
    first = np.cumsum(held) - held
    where = np.concatenate([np.arange(n, n + m) for n, m in zip(lens, new)])
    at = torch.from_numpy(np.concatenate([f + np.arange(n, n + m) // page for f, n, m in zip(first, lens, new)])).cuda()
    rows = len(where)
    s.update(position=torch.from_numpy(where).to(torch.int32).cuda(),
             slot=perm[at] * page + torch.from_numpy(where % page).cuda(),
             k_cache=_normal((pool, page, H, D), ct, g), v_cache=_normal((pool, page, H, D), ct, g),
             q=_normal((rows, case["heads"], D), dt, g) if case["queries"] else None,
             k=_normal((rows, H, D), dt, g), v=_normal((rows, H, D), dt, g))
    s["k_scale"], s["v_scale"] = _scales(case, g)
    s["out"] = torch.zeros_like(s["q"]) if case["queries"] else None
    f = _frequencies(case)
    s["freq"] = torch.from_numpy(f).cuda()
    if own:
        sv = _package()
        s["turns"] = sv.rope_table(f) if case["rotary"] else None
        s["ws"] = sv.alloc_cache_workspace(B)
    return s


# ----------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"shared": _shared_own, "plan": _plan_own, "map": _map_own, "rows": _rows_own}[op](state)
    return {"shared": _shared_plain, "plan": _plan_plain, "map": _map_plain, "rows": _rows_plain}[op](state)


def _plan_own(s):
    c = s["case"]
    _package().share_plan(s["table"], s["cache_len"], s["verify_len"], s["row"], gamma=c["gamma"], rows=s["rows"],
                          page_size=c["page"], least=LEAST, out_leader=s["leader"], out_shared=s["shared"],
                          plan=s["plan"])
    return dict(leader=s["leader"], shared=s["shared"])


def _shared_own(s):
    """A round's plan, and the attention of its layers."""
    c = s["case"]
    sv = _package()
    _plan_own(s)
    for i in range(c["layers"]):
        sv.attend_shared(s["q"][i], s["k_cache"][i], s["v_cache"][i], s["table"], s["plan"], gamma=c["gamma"],
                         k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"][i], workspace=s["ws"])
    return s["out"]


def _map_own(s):
    """The new rows' pages and slots; then the rows are given up again (an accept
    length of -1), so that a pass leaves the state as it found it."""
    c = s["case"]
    sv = _package()
    sv.map_rows(s["table"], s["num"], s["ref"], s["cache_len"], s["new_len"], rows=s["rows"], page_size=c["page"],
                out_first=s["first"], out_request=s["request"], out_position=s["position"], out_slot=s["slot"],
                out_status=s["status"], workspace=s["ws"])
    grown, held = s["table"].clone(), s["num"].clone()
    sv.commit_pages(s["table"], s["num"], s["ref"], s["cache_len"], s["none"], page_size=c["page"], workspace=s["ws"])
    return dict(table=grown, num=held, first=s["first"], request=s["request"], position=s["position"], slot=s["slot"],
                status=s["status"], ref=s["ref"])


def _rows_own(s):
    c = s["case"]
    _package().append_rows(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["position"], s["slot"],
                           turns=s["turns"], interleaved=c["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                           out_q=s["out"], workspace=s["ws"])
    out = dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    return dict(q=s["out"], **out) if c["queries"] else out


# ------------------------------------------------------------- plain forms
def _plan_plain(s):
    """Requests that begin with the same page are compared with the lowest of
    them; the leading pages that save most, and who has them, become a group; the
    others go into the next pass."""
    c = s["case"]
    table, B = s["table"], c["B"]
    slots = table.shape[1]
    full = (s["cache_len"] // c["page"]).long()
    me = torch.arange(B, device="cuda")
    left = (full > 0) & (table[:, 0] >= 0)
    leader, shared = me.clone(), torch.zeros_like(me)
    lower = me[None, :] < me[:, None]
    for _ in range(PASSES):
        same = left[:, None] & left[None, :] & (table[:, 0][:, None] == table[:, 0][None, :])
        head = torch.where(left, torch.where(same & lower, me[None, :], me[:, None]).amin(1), me)
        alike = (table == table[head]) & (table >= 0) & \
            (torch.arange(slots, device="cuda")[None, :] < torch.minimum(full, full[head])[:, None])
        depth = alike.to(torch.int32).cumprod(1).sum(1)
        depth = torch.where(left, depth, 0)
        count = (same & (depth[None, :] >= depth[:, None])).sum(1)
        worth = left & (head != me) & (depth * c["page"] >= LEAST)
        gain = torch.where(worth, (count - 1) * depth, 0)
        # the largest gain of each class, ties to the larger group
        key = gain * 8192 + torch.where(worth, count, 0)
        best = torch.where(same, key[None, :], 0).amax(1)
        got = best // 8192
        d = torch.where(got > 0, got // (best % 8192 - 1).clamp(min=1), 0)
        joins = left & (got > 0) & (depth >= d)
        leader = torch.where(joins, head, leader)
        shared = torch.where(joins, d, shared)
        left = left & ~joins & (head != me)
    s["leader"].copy_(leader)
    s["shared"].copy_(shared)
    return dict(leader=s["leader"], shared=s["shared"])


def _gather(cache, table):
    """[B, slots * page, H, D] in 32 bits."""
    if cache.dtype == torch.float8_e4m3fn:
        x = cache.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
    else:
        x = cache[table].float()
    return x.flatten(1, 2)


def _put(out, at, has, values):
    """`out` with the rows that exist set, the others as they were."""
    flat = out.view(-1, *out.shape[-2:])
    spare = torch.cat([flat, flat[:1]])
    spare[torch.where(has, at, flat.shape[0])] = values.to(out.dtype)
    flat.copy_(spare[:-1])


def _shared_plain(s):
    c = s["case"]
    B, G1, H, D = c["B"], c["gamma"] + 1, c["kv_heads"], c["dim"]
    group = c["heads"] // H
    j = torch.arange(G1, device="cuda")[None, :]
    has = (j <= (s["verify_len"][:, None] if s["verify_len"] is not None else c["gamma"])).expand(B, G1)
    base = s["row"].long()[:, None] if c["packed"] else torch.arange(B, device="cuda")[:, None] * G1
    at = torch.where(has, base + j, 0)
    table = s["table"].clamp(min=0).long()
    for i in range(c["layers"]):
        K = _gather(s["k_cache"][i], table).permute(0, 2, 3, 1)  # [B, H, D, L]
        q = s["q"][i].reshape(-1, c["heads"], D)[at].float()
        q = q.view(B, G1, H, group, D).permute(0, 2, 1, 3, 4).reshape(B, H, G1 * group, D)
        x = torch.matmul(q, K) * (1.0 / math.sqrt(D))
        del K
        if s["k_scale"] is not None:
            x = x * s["k_scale"][None, :, None, None]
        t = torch.arange(x.shape[-1], device="cuda")[None, None, :]
        p = (s["cache_len"].long()[:, None] + torch.arange(G1, device="cuda"))[:, :, None]
        x = x.view(B, H, G1, group, -1).masked_fill(~(t <= p)[:, None, :, None, :], -math.inf)
        w = torch.exp(x - x.amax(-1, keepdim=True))
        del x
        total = w.sum(-1, keepdim=True)
        V = _gather(s["v_cache"][i], table).transpose(1, 2)  # [B, H, L, D]
        o = torch.matmul(w.view(B, H, G1 * group, -1), V).view(B, H, G1, group, D) / total
        del w, V
        if s["v_scale"] is not None:
            o = o * s["v_scale"][None, :, None, None, None]
        _put(s["out"][i], at, has, o.permute(0, 2, 1, 3, 4).reshape(B, G1, c["heads"], D))
    return s["out"]


def _map_plain(s):
    c = s["case"]
    page, table, num, ref = c["page"], s["table"], s["num"], s["ref"]
    one = torch.ones((), dtype=torch.int32, device="cuda")
    n, m = s["cache_len"], s["new_len"]
    grow = ((n + m + page - 1) // page - num).clamp(min=0)
    upto = torch.cumsum(grow, 0)
    fits = (upto <= (ref == 0).sum()) | (grow == 0)
    free = torch.argsort((ref != 0).to(torch.uint8), stable=True)
    slot = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (slot >= num[:, None]) & (slot < (num + grow)[:, None]) & fits[:, None]
    rank = torch.where(fresh, (upto - grow)[:, None] + slot - num[:, None], 0).clamp(max=ref.numel() - 1)
    table.copy_(torch.where(fresh, free[rank].to(torch.int32), table))
    ref.index_add_(0, table.clamp(min=0).view(-1).long(), torch.where(fresh, one, 0 * one).view(-1))
    num.copy_(torch.where(fits, num + grow, num))
    s["status"].copy_(torch.where(fits, 0, -15))
    # the rows, one request's behind the other's
    s["first"][1:] = torch.cumsum(m, 0)
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["first"][1:].long(), r, right=True).clamp(max=c["B"] - 1)
    pos = (n.long()[b] + r - s["first"].long()[b])
    entry = table[b, (pos // page).clamp(max=table.shape[1] - 1)].long()
    s["request"].copy_(b)
    s["position"].copy_(pos)
    s["slot"].copy_(torch.where(fits[b], entry * page + pos % page, -1))
    grown, held = table.clone(), num.clone()
    # what is behind the cache's end is given back
    keep = (n + page - 1) // page
    drop = (slot >= keep[:, None]) & (slot < num[:, None])
    ref.index_add_(0, table.clamp(min=0).view(-1).long(), torch.where(drop, -one, 0 * one).view(-1))
    table.masked_fill_(drop, -1)
    num.copy_(torch.minimum(num, keep))
    return dict(table=grown, num=held, first=s["first"], request=s["request"], position=s["position"], slot=s["slot"],
                status=s["status"], ref=ref)


def _turned(x, cos, sin, interleaved):
    """The rotated x [rows, heads, D] in 32 bits; cos, sin [rows, 1, rotary / 2]."""
    half = cos.shape[-1]
    x = x.float()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _rows_plain(s):
    c = s["case"]
    H, D = c["kv_heads"], c["dim"]
    angle = s["position"].double()[:, None] * s["freq"]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    new = _turned(s["k"], cos, sin, c["interleaved"]), s["v"].float()
    for cache, x, scale in zip((s["k_cache"], s["v_cache"]), new, (s["k_scale"], s["v_scale"])):
        if scale is not None:
            x = (x / scale[:, None]).clamp(-448.0, 448.0)
        x = x.to(cache.dtype)
        flat = cache.view(-1, H, D)
        if cache.dtype == torch.float8_e4m3fn:
            flat, x = flat.view(torch.uint8), x.view(torch.uint8)
        flat[s["slot"]] = x
    out = dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    if not c["queries"]:
        return out
    s["out"].copy_(_turned(s["q"], cos, sin, c["interleaved"]))
    return dict(q=s["out"], **out)


# ------------------------------------------------------------ from the definition
def exact(case, seed):
    s = prepare(case, seed)
    return {"shared": _shared_exact, "plan": _plan_exact, "map": _map_exact, "rows": _rows_exact}[case["op"]](s)


def _plan_exact(s):
    """By hand: classes of requests with the same first page, one leader after the other."""
    c = s["case"]
    table, lens = s["table"].tolist(), s["cache_len"].tolist()
    full = [n // c["page"] for n in lens]
    leader, shared = list(range(c["B"])), [0] * c["B"]

    def common(a, b):
        n = 0
        while n < min(full[a], full[b]) and table[a][n] == table[b][n] >= 0:
            n += 1
        return n

    classes = {}
    for b in range(c["B"]):
        if full[b] > 0 and table[b][0] >= 0:
            classes.setdefault(table[b][0], []).append(b)
    for members in classes.values():
        for _ in range(PASSES):
            if not members:
                break
            head, rest = members[0], members[1:]
            depth = {b: common(head, b) for b in rest}
            options = []
            for d in set(depth.values()):
                others = sum(x >= d for x in depth.values())
                if d * c["page"] >= LEAST:
                    options.append((others * d, others, d))
            _, _, d = max(options, default=(0, 0, 0))
            if d:
                leader[head], shared[head] = head, d
                for b in rest:
                    if depth[b] >= d:
                        leader[b], shared[b] = head, d
            members = [b for b in rest if not d or depth[b] < d]
    return dict(leader=_ints(leader), shared=_ints(shared))


def _shared_exact(s):
    """One request and KV head at a time, over the keys that it has."""
    c = s["case"]
    lens = s["cache_len"].tolist()
    ell = s["verify_len"].tolist() if s["verify_len"] is not None else [c["gamma"]] * c["B"]
    H, D, page = c["kv_heads"], c["dim"], c["page"]
    group = c["heads"] // H
    if c["layers"] * 4 * D * c["heads"] * sum((n + e + 1) * (e + 1) for n, e in zip(lens, ell)) > 2e12:
        return None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for i in range(c["layers"]):
        rows, q = out[i].view(-1, c["heads"], D), s["q"][i].view(-1, c["heads"], D)
        k, v = s["k_cache"][i], s["v_cache"][i]
        first = 0
        for b, (n, e) in enumerate(zip(lens, ell)):
            base = first if c["packed"] else b * (c["gamma"] + 1)
            first += e + 1
            at = torch.arange(n + e + 1, device="cuda")
            pages, off = s["table"][b, at // page].long(), at % page
            hidden = torch.arange(n, n + e + 1, device="cuda")[:, None] < at[None, :]
            for h in range(H):
                K, V = ((x[:, :, h].view(torch.uint8)[pages, off].view(x.dtype) if c["cache"] == "e4m3"
                         else x[pages, off, h]).double() for x in (k, v))
                if s["k_scale"] is not None:
                    K, V = K * s["k_scale"][h].double(), V * s["v_scale"][h].double()
                Q = q[base:base + e + 1, h * group:(h + 1) * group].double()
                x = torch.einsum("rgd,td->rgt", Q, K) / math.sqrt(D)
                x = torch.where(hidden[:, None, :], torch.full_like(x, -math.inf), x)
                rows[base:base + e + 1, h * group:(h + 1) * group] = \
                    torch.einsum("rgt,td->rgd", torch.softmax(x, -1), V)
    return out


def _map_exact(s):
    """The pages by hand, request after request."""
    c = s["case"]
    page = c["page"]
    table, num, ref, lens, new = (s[k].tolist() for k in ("table", "num", "ref", "cache_len", "new_len"))
    before = list(ref)
    free = [i for i, n in enumerate(ref) if n == 0]
    taken, closed = 0, False
    status, first, request, position, slot = [], [0], [], [], []
    for b, (n, m) in enumerate(zip(lens, new)):
        grow = max(0, _pages(n + m, page) - num[b])
        closed = closed or taken + grow > len(free)
        ok = grow == 0 or not closed
        if ok:
            for p in free[taken:taken + grow]:
                table[b][num[b]] = p
                num[b] += 1
            taken += grow
        status.append(0 if ok else -15)
        request += [b] * m
        position += range(n, n + m)
        slot += [table[b][t // page] * page + t % page for t in range(n, n + m)] if ok else [-1] * m
        first.append(first[-1] + m)
    return dict(table=_ints(table), num=_ints(num), first=_ints(first), request=_ints(request),
                position=_ints(position), slot=torch.tensor(slot, dtype=torch.int64, device="cuda"),
                status=_ints(status), ref=_ints(before))


def _rows_exact(s):
    """Complex rotation in 64 bits."""
    c = s["case"]
    H, D, half = c["kv_heads"], c["dim"], c["rotary"] // 2
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    freq = torch.from_numpy(_frequencies(c)).cuda()

    def turned(x):
        x = x.double().clone()
        if half:
            z = x[..., :2 * half].unflatten(-1, (half, 2)) if c["interleaved"] else \
                x[..., :2 * half].unflatten(-1, (2, half)).transpose(-1, -2)
            turn = torch.polar(torch.ones_like(freq), s["position"].double()[:, None] * freq)[:, None]
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            x[..., :2 * half] = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return x

    for cache, x, scale in zip(caches, (turned(s["k"]), s["v"].double()), (s["k_scale"], s["v_scale"])):
        if scale is not None:
            x = (x / scale.double()[:, None]).clamp(-448.0, 448.0)
        cache.view(-1, H, D)[s["slot"]] = x
    out = dict(k_cache=caches[0], v_cache=caches[1])
    return dict(q=turned(s["q"]), **out) if c["queries"] else out
