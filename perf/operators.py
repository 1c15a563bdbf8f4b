"""Cases that measure the paged key-value cache operators: attention of the
tested tokens over the cache, rotary positions with the append, and the page
operations of a verification round (reserve, commit, fork, compact).

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


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token for a handful of chats: the latency of one decoding step
        dict(name="attend_one_token_small", op="attend", B=4, gamma=0, heads=32, kv_heads=8, dim=128, page=16,
             shortest=1, longest=1024, dtype="bf16", cache="bf16", window=0, sinks=0, packed=False, full=True),
        # one new token for each of 32 long documents of uneven lengths: the cache's bandwidth
        dict(name="attend_one_token_long", op="attend", B=32, gamma=0, heads=32, kv_heads=8, dim=128, page=64,
             shortest=2000, longest=32768, dtype="bf16", cache="bf16", window=0, sinks=0, packed=False, full=True),
        # blocks of 16 drafts verified at once (the block-diffusion workload's batch and block)
        dict(name="attend_verify_block", op="attend", B=64, gamma=16, heads=32, kv_heads=8, dim=128, page=64,
             shortest=500, longest=8192, dtype="bf16", cache="bf16", window=0, sinks=0, packed=False, full=True),
        # scheduled ragged lengths in packed rows, sliding window with sinks, 8-bit cache, an odd group of heads
        dict(name="attend_verify_window_e4m3", op="attend", B=64, gamma=16, heads=28, kv_heads=4, dim=64, page=16,
             shortest=1, longest=12000, dtype="fp16", cache="e4m3", window=4000, sinks=4, packed=True, full=False),
        # a chat batch's new keys: half layout over the whole head
        dict(name="append_small", op="append", B=16, gamma=4, heads=32, kv_heads=8, dim=128, rotary=128, page=16,
             shortest=1, longest=4096, dtype="bf16", cache="bf16", interleaved=False, scaling="none", packed=False,
             full=True),
        # a large batch of drafted blocks at far positions, interleaved pairs in half of the head, scaled, 8-bit cache
        dict(name="append_large", op="append", B=512, gamma=16, heads=32, kv_heads=8, dim=128, rotary=64, page=32,
             shortest=1, longest=1000, dtype="bf16", cache="e4m3", interleaved=True, scaling="banded", packed=True,
             full=False),
        # pages taken for the drafts and given back after the accept lengths are known
        dict(name="round_small", op="round", B=16, gamma=4, page=16, shortest=1, longest=2000, spare=200, window=0,
             sinks=0),
        dict(name="round_large", op="round", B=1024, gamma=16, page=16, shortest=1, longest=6000, spare=60000,
             window=0, sinks=0),
        # one prompt sampled four times; and half of a batch branching into the other half
        dict(name="fork_small", op="fork", B=5, sources=1, forks=4, layers=2, kv_heads=8, dim=128, page=16,
             shortest=300, longest=900, cache="bf16", spare=16),
        dict(name="fork_large", op="fork", B=128, sources=64, forks=64, layers=8, kv_heads=8, dim=128, page=64,
             shortest=1, longest=500, cache="bf16", spare=100),
        # a pool with holes after requests have ended
        dict(name="compact_small", op="compact", B=8, layers=2, kv_heads=8, dim=64, page=16, shortest=1, longest=300,
             cache="e4m3", holes=0.5),
        dict(name="compact_large", op="compact", B=64, layers=4, kv_heads=8, dim=128, page=32, shortest=100,
             longest=1500, cache="bf16", holes=0.7),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "round", "fork", "compact"])
    page = rng.choice([1, 5, 8, 16, 16, 32, 48, 64, 64, 128, 256])
    if op == "attend":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        gamma = rng.choice([0, 0, 1, 3, 4, 7, 8, 13, 16, 32])
        kv_heads = rng.choice([1, 2, 4, 5, 8])
        group = rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
        dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
        B = _log(rng, 1, 96)
        # bounded so that no drawn case has more keys, or more work per key, than the largest listed ones
        longest = min(_log(rng, 16, 40000), max(16, 500_000_000 // (B * kv_heads * dim)),
                      max(16, 16_000_000_000 // (B * kv_heads * group * (gamma + 1) * dim)))
        if dtype == "fp32":
            longest = max(8, longest // 4)
        window = rng.choice([0, 0, 0, _log(rng, 1, longest)])
        return dict(op=op, B=B, gamma=gamma, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page,
                    shortest=_log(rng, 1, longest), longest=longest, dtype=dtype,
                    cache=dtype if dtype == "fp32" else rng.choice([dtype, dtype, "e4m3"]), window=window,
                    sinks=rng.choice([0, 1, 4, 17]) if window else 0, packed=rng.random() < 0.5,
                    full=rng.random() < 0.5)
    if op == "append":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        kv_heads = rng.choice([1, 2, 4, 5, 8])
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        B = _log(rng, 1, 512)
        gamma = rng.choice([0, 0, 1, 4, 8, 16, 32])
        group = rng.choice([1, 2, 4, 7])
        while B * (gamma + 1) * kv_heads * (group + 2) * dim > 512 * 9 * 48 * 128:
            B = B // 2
        longest = min(_log(rng, 16, 200000), max(16, 60_000_000 // (B * kv_heads * dim)))
        return dict(op=op, B=B, gamma=gamma, heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    rotary=rng.choice([dim, dim, dim // 2, dim // 4]), page=page, shortest=_log(rng, 1, longest),
                    longest=longest, dtype=dtype,
                    cache=dtype if dtype == "fp32" else rng.choice([dtype, dtype, "e4m3"]),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "banded"]),
                    packed=rng.random() < 0.5, full=rng.random() < 0.5)
    if op == "round":
        B = _log(rng, 1, 1024)
        longest = _log(rng, 8, 6000)
        window = rng.choice([0, 0, _log(rng, 1, longest)])
        if page == 1:
            longest = min(longest, 1500)
        return dict(op=op, B=B, gamma=rng.choice([0, 1, 4, 8, 16, 32]), page=page, shortest=_log(rng, 1, longest),
                    longest=longest, spare=_log(rng, 40 * B, 60 * B + 100), window=window,
                    sinks=rng.choice([0, 4, 33]) if window else 0)
    kv_heads = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 80, 128, 128, 256])
    cache = rng.choice(["bf16", "fp16", "fp32", "e4m3"])
    layers = rng.choice([1, 2, 4, 7])
    per_token = layers * kv_heads * dim * SIZE[cache]
    B = _log(rng, 2, 96)
    longest = max(4, min(_log(rng, 16, 1500), 150_000_000 // (per_token * B)))
    page = min(page, 64)
    if op == "fork":
        sources = rng.randint(1, max(1, B // 2))
        return dict(op=op, B=B, sources=sources, forks=rng.randint(1, B - sources), layers=layers, kv_heads=kv_heads,
                    dim=dim, page=page, shortest=_log(rng, 1, longest), longest=longest, cache=cache, spare=B + 3)
    return dict(op=op, B=B, layers=layers, kv_heads=kv_heads, dim=dim, page=page, shortest=_log(rng, 1, longest),
                longest=longest, cache=cache, holes=rng.choice([0.1, 0.3, 0.5, 0.8]))


# ------------------------------------------------------- lengths (by the case)
def _lengths(case):
    """The requests' cache lengths, verify lengths and accept lengths: they
    belong to the case, so that every seed has the same work."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    B, gamma = case["B"], case.get("gamma", 0)
    lo, hi = case["shortest"], max(case["longest"], case["shortest"])
    lens = [r.randint(lo, hi) for _ in range(B)]
    lens[r.randrange(B)] = hi
    ell = [gamma if case.get("full", False) else r.randint(0, gamma) for _ in range(B)]
    acc = [r.randint(0, n) for n in ell]
    return lens, ell, acc


def _pages(n, page):
    return -(-n // page)


def _seen(n, ell, window, sinks):
    """Keys that the tokens at positions n .. n + ell see between them, and the
    pairs of token and key."""
    if not window:
        return n + ell + 1, sum(n + j + 1 for j in range(ell + 1))
    first = max(0, n - window + 1)
    union = n + ell + 1 - first + min(sinks, first)
    pairs = 0
    for j in range(ell + 1):
        f = max(0, n + j - window + 1)
        pairs += n + j + 1 - f + min(sinks, f)
    return union, pairs


def work(case):
    lens, ell, _ = _lengths(case)
    op = case["op"]
    if op == "attend":
        per_key = 2 * case["kv_heads"] * case["dim"] * SIZE[case["cache"]]
        rows = sum(e + 1 for e in ell)
        seen = [_seen(n, e, case["window"], case["sinks"]) for n, e in zip(lens, ell)]
        return dict(bytes=sum(s[0] for s in seen) * per_key + 2 * rows * case["heads"] * case["dim"] * SIZE[case["dtype"]]
                    + 4 * sum(_pages(n + e + 1, case["page"]) for n, e in zip(lens, ell)),
                    flops=4 * case["dim"] * case["heads"] * sum(s[1] for s in seen))
    if op == "append":
        rows = sum(e + 1 for e in ell)
        es, cs = SIZE[case["dtype"]], SIZE[case["cache"]]
        return dict(bytes=rows * case["dim"] * (2 * case["heads"] * es + 2 * case["kv_heads"] * (es + cs)),
                    flops=3 * rows * case["rotary"] * (case["heads"] + case["kv_heads"]))
    if op == "round":
        # the references of the pool are read once (to find the free pages); lengths and new entries
        pool = sum(_pages(n, case["page"]) for n in lens) + case["spare"]
        return dict(bytes=4 * pool + 4 * case["B"] * 8, flops=0)
    per_token = 2 * case["layers"] * case["kv_heads"] * case["dim"] * SIZE[case["cache"]]
    if op == "fork":
        copied = sum(lens[i % case["sources"]] % case["page"] for i in range(case["forks"]))
        shared = sum(_pages(lens[i % case["sources"]], case["page"]) for i in range(case["forks"]))
        return dict(bytes=2 * copied * per_token + 12 * shared, flops=0)
    live, pool = _compact_pool(case)
    movers = max(1.0, live * (1.0 - live / pool))  # expected number of live pages behind the first `live` ids
    return dict(bytes=2 * movers * case["page"] * per_token + 8 * pool + 8 * live, flops=0)


def _compact_pool(case):
    lens, _, _ = _lengths(case)
    live = sum(_pages(n, case["page"]) for n in lens)
    return live, int(math.ceil(live / (1.0 - case["holes"]))) + 1


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


def _table(held, slots, pool, g):
    """Pages of each request, drawn from the pool without order: [B, slots], -1 behind the last."""
    perm = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    held_t = torch.tensor(held, device="cuda")
    start = torch.cumsum(held_t, 0) - held_t
    at = torch.arange(slots, device="cuda")[None, :]
    return torch.where(at < held_t[:, None], perm[(start[:, None] + at).clamp(max=pool - 1)],
                       torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()


def _frequencies(case):
    """Angle per token of each rotated pair (64 bits): base 10000, or 500000 where the context is scaled; "linear"
    divides every frequency by 4; "banded" divides by 8 those with a wave over 8192 tokens, none with one under
    2048, and blends in between."""
    half = case["rotary"] // 2
    base = 10000.0 if case["scaling"] == "none" else 500000.0
    f = base ** (-np.arange(half, dtype=np.float64) / half)
    if case["scaling"] == "linear":
        f = f / 4.0
    if case["scaling"] == "banded":
        wave = 2.0 * math.pi / f
        blend = np.clip((8192.0 / wave - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = (1.0 - blend) * f / 8.0 + blend * f
    return f


def prepare(case, seed):
    lens, ell, acc = _lengths(case)
    B, op, page = case["B"], case["op"], case["page"]
    g = _gen(seed, 1)
    s = dict(case=case)
    if op in ("attend", "append"):
        held = [_pages(n + e + 1, page) for n, e in zip(lens, ell)]
        pool = sum(held) + 3
        H, D = case["kv_heads"], case["dim"]
        dt, ct = TYPES[case["dtype"]], TYPES[case["cache"]]
        s.update(table=_table(held, max(held), pool, g), cache_len=_ints(lens),
                 verify_len=None if case["full"] else _ints(ell), row=None, k_scale=None, v_scale=None,
                 k_cache=_normal((pool, page, H, D), ct, g), v_cache=_normal((pool, page, H, D), ct, g))
        if case["cache"] == "e4m3":
            s["k_scale"] = torch.rand(H, device="cuda", generator=g) * 0.05 + 0.02
            s["v_scale"] = torch.rand(H, device="cuda", generator=g) * 0.05 + 0.02
            if op == "attend":  # entries as a quantised cache holds them: well inside the type's range
                s["k_cache"] = _normal((pool, page, H, D), ct, g, 20.0)
                s["v_cache"] = _normal((pool, page, H, D), ct, g, 20.0)
        rows = (sum(e + 1 for e in ell),) if case["packed"] else (B, case["gamma"] + 1)
        if case["packed"]:
            n = np.array([e + 1 for e in ell])
            s["row"] = _ints((np.cumsum(n) - n).tolist())
        std = 2.0 if op == "attend" else 1.0
        s["q"] = _normal(rows + (case["heads"], D), dt, g, std)
        s["out"] = torch.zeros_like(s["q"])
        if op == "append":
            s["k"] = _normal(rows + (H, D), dt, g)
            s["v"] = _normal(rows + (H, D), dt, g)
            f = _frequencies(case)
            s["freq"] = torch.from_numpy(f).cuda()
            if own:
                import speculative_decoding_verification_softmax_gb300 as sv
                s["turns"] = sv.rope_table(f)
        if own:
            import speculative_decoding_verification_softmax_gb300 as sv
            s["ws"] = (sv.alloc_attend_workspace(B, case["gamma"], case["heads"], H, D) if op == "attend"
                       else sv.alloc_cache_workspace(B))
        return s
    if op == "round":
        # the committed lengths' pages are held already, as after the round before
        w, sk = case["window"], case["sinks"]
        held = [_pages(n + a + 1, page) for n, a in zip(lens, acc)]
        most = max(_pages(n + case["gamma"] + 1, page) for n in lens)
        pool = sum(held) + case["spare"]
        table = _table(held, most, pool, g)
        if w:  # pages behind the window have been given back
            first = torch.arange(most, device="cuda")[None, :] * page
            new_len = (_ints(lens) + _ints(acc) + 1)[:, None]
            gone = (first >= sk) & (first + page <= new_len - w + 1)
            table = torch.where(gone, torch.full_like(table, -1), table)
        ref = torch.zeros(pool + 1, dtype=torch.int32, device="cuda")
        ref.index_add_(0, torch.where(table < 0, pool, table).view(-1).long(), torch.ones(table.numel(), dtype=torch.int32, device="cuda"))
        s.update(table=table, num=_ints(held), ref=ref[:pool].contiguous(), cache_len=_ints(lens),
                 verify_len=_ints(ell), accept=_ints(acc), new_len=torch.zeros(B, dtype=torch.int32, device="cuda"),
                 status=torch.zeros(B, dtype=torch.int32, device="cuda"))
    else:
        H, D, L, ct = case["kv_heads"], case["dim"], case["layers"], TYPES[case["cache"]]
        if op == "fork":
            held = [_pages(n, page) if b < case["sources"] else 0 for b, n in enumerate(lens)]
            pool, slots = sum(held) + case["spare"], max(_pages(n, page) for n in lens)
            lens = [n if b < case["sources"] else 0 for b, n in enumerate(lens)]
            s.update(src=_ints([i % case["sources"] for i in range(case["forks"])]),
                     dst=_ints([case["sources"] + i for i in range(case["forks"])]),
                     status=torch.zeros(case["forks"], dtype=torch.int32, device="cuda"))
        else:
            held = [_pages(n, page) for n in lens]
            pool, slots = _compact_pool(case)[1], max(held)
        table = _table(held, slots, pool, g)
        ref = torch.zeros(pool + 1, dtype=torch.int32, device="cuda")
        ref.index_add_(0, torch.where(table < 0, pool, table).view(-1).long(), torch.ones(table.numel(), dtype=torch.int32, device="cuda"))
        s.update(table=table, num=_ints(held), ref=ref[:pool].contiguous(), cache_len=_ints(lens),
                 k_cache=_normal((L, pool, page, H, D), ct, g), v_cache=_normal((L, pool, page, H, D), ct, g))
        if op == "compact":
            s.update(out_table=torch.zeros_like(table), out_ref=torch.zeros_like(s["ref"]))
    if own:
        import speculative_decoding_verification_softmax_gb300 as sv
        s["ws"] = sv.alloc_cache_workspace(B, s["ref"].numel())
    return s


# ----------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _attend_own, "append": _append_own, "round": _round_own, "fork": _fork_own,
                "compact": _compact_own}[op](state)
    return {"attend": _attend_plain, "append": _append_plain, "round": _round_plain, "fork": _fork_plain,
            "compact": _compact_plain}[op](state)


def _attend_own(s):
    import speculative_decoding_verification_softmax_gb300 as sv
    c = s["case"]
    sv.attend(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cache_len"], s["verify_len"], s["row"],
              gamma=c["gamma"], window=c["window"], sinks=c["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"],
              out=s["out"], workspace=s["ws"])
    return s["out"]


def _append_own(s):
    import speculative_decoding_verification_softmax_gb300 as sv
    c = s["case"]
    sv.append_kv(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cache_len"], s["verify_len"],
                 s["row"], gamma=c["gamma"], turns=s["turns"], interleaved=c["interleaved"], k_scale=s["k_scale"],
                 v_scale=s["v_scale"], out_q=s["out"], workspace=s["ws"])
    return dict(q=s["out"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _round_own(s):
    import speculative_decoding_verification_softmax_gb300 as sv
    c = s["case"]
    sv.reserve_pages(s["table"], s["num"], s["ref"], s["cache_len"], s["verify_len"], gamma=c["gamma"],
                     page_size=c["page"], out_status=s["status"], workspace=s["ws"])
    reserved = s["table"].clone()
    sv.commit_pages(s["table"], s["num"], s["ref"], s["cache_len"], s["accept"], page_size=c["page"],
                    window=c["window"], sinks=c["sinks"], out_cache_len=s["new_len"], workspace=s["ws"])
    return dict(reserved=reserved, table=s["table"], num=s["num"], ref=s["ref"], new_len=s["new_len"],
                status=s["status"])


def _fork_own(s):
    import speculative_decoding_verification_softmax_gb300 as sv
    sv.fork_pages(s["table"], s["num"], s["ref"], s["cache_len"], s["src"], s["dst"], s["k_cache"], s["v_cache"],
                  out_status=s["status"], workspace=s["ws"])
    return {k: s[k] for k in ("table", "num", "ref", "cache_len", "k_cache", "v_cache", "status")}


def _compact_own(s):
    import speculative_decoding_verification_softmax_gb300 as sv
    total, _ = sv.compact_pages(s["table"], s["num"], s["ref"], s["k_cache"], s["v_cache"],
                                out_page_table=s["out_table"], out_ref_count=s["out_ref"], workspace=s["ws"])
    return dict(table=s["out_table"], ref=s["out_ref"], total=total, k_cache=s["k_cache"], v_cache=s["v_cache"])


# ------------------------------------------------------------- plain forms
def _rows(s):
    """[B, gamma+1] rows of q, and which of them the request has."""
    c = s["case"]
    j = torch.arange(c["gamma"] + 1, device="cuda")[None, :]
    ell = s["verify_len"][:, None] if s["verify_len"] is not None else c["gamma"]
    has = (j <= ell).expand(c["B"], c["gamma"] + 1)
    if c["packed"]:
        at = s["row"].long()[:, None] + j
    else:
        at = (torch.arange(c["B"], device="cuda")[:, None] * (c["gamma"] + 1)) + j
    return torch.where(has, at, 0), has


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
    return out


def _attend_plain(s):
    c = s["case"]
    B, G1, H, D = c["B"], c["gamma"] + 1, c["kv_heads"], c["dim"]
    group = c["heads"] // H
    at, has = _rows(s)
    table = s["table"].clamp(min=0).long()
    K = _gather(s["k_cache"], table).permute(0, 2, 3, 1)  # [B, H, D, L]
    q = s["q"].reshape(-1, c["heads"], D)[at].float()  # [B, G1, heads, D]
    q = q.view(B, G1, H, group, D).permute(0, 2, 1, 3, 4).reshape(B, H, G1 * group, D)
    x = torch.matmul(q, K) * (1.0 / math.sqrt(D))
    del K
    if s["k_scale"] is not None:
        x = x * s["k_scale"][None, :, None, None]
    t = torch.arange(x.shape[-1], device="cuda")[None, None, :]
    p = (s["cache_len"].long()[:, None] + torch.arange(G1, device="cuda"))[:, :, None]
    see = t <= p
    if c["window"]:
        see = see & ((p - t < c["window"]) | (t < c["sinks"]))
    see = see[:, None, :, None, :]
    x = x.view(B, H, G1, group, -1).masked_fill(~see, -math.inf)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    del x
    total = w.sum(-1, keepdim=True)
    V = _gather(s["v_cache"], table).transpose(1, 2)  # [B, H, L, D]
    o = torch.matmul(w.view(B, H, G1 * group, -1), V).view(B, H, G1, group, D) / total
    if s["v_scale"] is not None:
        o = o * s["v_scale"][None, :, None, None, None]
    return _put(s["out"], at, has, o.permute(0, 2, 1, 3, 4).reshape(B, G1, c["heads"], D))


def _turned(x, cos, sin, interleaved):
    """The rotated x [..., heads, D] in 32 bits; cos, sin [..., 1, rotary / 2]."""
    half = cos.shape[-1]
    x = x.float()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _append_plain(s):
    c = s["case"]
    B, G1, H, D, page = c["B"], c["gamma"] + 1, c["kv_heads"], c["dim"], c["page"]
    at, has = _rows(s)
    pos = s["cache_len"].long()[:, None] + torch.arange(G1, device="cuda")
    angle = pos.double()[:, :, None] * s["freq"]
    cos, sin = angle.cos().float()[:, :, None, :], angle.sin().float()[:, :, None, :]
    q = _turned(s["q"].reshape(-1, c["heads"], D)[at], cos, sin, c["interleaved"])
    k = _turned(s["k"].reshape(-1, H, D)[at], cos, sin, c["interleaved"])
    v = s["v"].reshape(-1, H, D)[at].float()
    _put(s["out"], at, has, q)
    slot = torch.where(has, pos // page, 0)
    entry = torch.gather(s["table"].long(), 1, slot) * page + pos % page
    for cache, x, scale in ((s["k_cache"], k, s["k_scale"]), (s["v_cache"], v, s["v_scale"])):
        flat = cache.view(-1, H, D)
        if scale is not None:
            x = (x / scale[:, None]).clamp(-448.0, 448.0)
        x = x.to(cache.dtype)
        if cache.dtype == torch.float8_e4m3fn:
            flat, x = flat.view(torch.uint8), x.view(torch.uint8)
        # rows that a request does not have write the first row's value again
        first = x[:, :1].expand(-1, G1, -1, -1)
        flat[torch.where(has, entry, entry[:, :1])] = torch.where(has[:, :, None, None], x, first)
    return dict(q=s["out"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _take(table, num, ref, need, wanted):
    """Lowest free pages for the requests of `wanted` whose pages fit, in order."""
    one = torch.ones((), dtype=torch.int32, device="cuda")
    grow = torch.where(wanted, (need - num).clamp(min=0), 0)
    upto = torch.cumsum(grow, 0)
    fits = (upto <= (ref == 0).sum()) | (grow == 0)
    free = torch.argsort((ref != 0).to(torch.uint8), stable=True)
    slot = torch.arange(table.shape[1], device="cuda")[None, :]
    new = (slot >= num[:, None]) & (slot < (num + grow)[:, None]) & fits[:, None]
    rank = torch.where(new, (upto - grow)[:, None] + slot - num[:, None], 0).clamp(max=ref.numel() - 1)
    table.copy_(torch.where(new, free[rank].to(torch.int32), table))
    ref.index_add_(0, table.clamp(min=0).view(-1).long(), torch.where(new, one, 0 * one).view(-1))
    num.copy_(torch.where(fits, num + grow, num))
    return fits


def _round_plain(s):
    c = s["case"]
    page, table, num, ref = c["page"], s["table"], s["num"], s["ref"]
    need = (s["cache_len"] + s["verify_len"] + page) // page
    fits = _take(table, num, ref, need, need <= table.shape[1])
    s["status"].copy_(torch.where(fits, 0, -15))
    reserved = table.clone()
    new_len = s["cache_len"] + s["accept"] + 1
    keep = (new_len + page - 1) // page
    slot = torch.arange(table.shape[1], device="cuda")[None, :]
    drop = slot >= keep[:, None]
    if c["window"]:
        first = slot * page
        drop = drop | ((first >= c["sinks"]) & (first + page <= new_len[:, None] - c["window"] + 1))
    drop = drop & (slot < num[:, None]) & (table >= 0)
    ref.index_add_(0, table.clamp(min=0).view(-1).long(), -drop.view(-1).to(torch.int32))
    table.masked_fill_(drop, -1)
    num.copy_(torch.minimum(num, keep))
    s["new_len"].copy_(new_len)
    return dict(reserved=reserved, table=table, num=num, ref=ref, new_len=s["new_len"], status=s["status"])


def _fork_plain(s):
    c = s["case"]
    page, table, num, ref, lens = c["page"], s["table"], s["num"], s["ref"], s["cache_len"]
    src, dst = s["src"].long(), s["dst"].long()
    slot = torch.arange(table.shape[1], device="cuda")[None, :]
    # the destinations give back what they hold
    old = table[dst]
    held = (slot < num[dst][:, None]) & (old >= 0)
    ref.index_add_(0, old.clamp(min=0).view(-1).long(), -held.view(-1).to(torch.int32))
    n = lens[src]
    tail, whole = n % page, n // page
    part = tail > 0
    free = torch.argsort((ref != 0).to(torch.uint8), stable=True)
    rank = torch.cumsum(part.to(torch.int32), 0) - 1
    fresh = free[rank.clamp(0, ref.numel() - 1)].to(torch.int32)
    fits = ~part | (rank < (ref == 0).sum())
    from_ = table[src]
    shared = (slot < whole[:, None]) & fits[:, None]
    last = (slot == whole[:, None]) & (part & fits)[:, None]
    rows = torch.where(shared, from_, torch.where(last, fresh[:, None], torch.full_like(from_, -1)))
    table[dst] = rows
    ref.index_add_(0, rows.clamp(min=0).view(-1).long(), (rows >= 0).view(-1).to(torch.int32))
    num[dst] = torch.where(fits, whole + part.to(torch.int32), 0)
    lens[dst] = torch.where(fits, n, 0)
    s["status"].copy_(torch.where(fits, 0, -15))
    source = torch.gather(from_, 1, whole.clamp(max=table.shape[1] - 1)[:, None].long())[:, 0].clamp(min=0)
    # a fork that copies nothing writes its source's last page onto itself
    for cache in (s["k_cache"], s["v_cache"]):
        x = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
        tokens = torch.where(part & fits, tail, 0)
        j = torch.arange(page, device="cuda")
        pages = torch.where(part & fits, fresh, source).long()
        take = (j[None, :] < tokens[:, None])[None, :, :, None, None]
        x[:, pages] = torch.where(take, x[:, source.long()], x[:, pages])
    return {k: s[k] for k in ("table", "num", "ref", "cache_len", "k_cache", "v_cache", "status")}


def _compact_plain(s):
    table, ref = s["table"], s["ref"]
    live = ref > 0
    pool = ref.numel()
    total = live.sum().to(torch.int32)
    at = torch.arange(pool, device="cuda", dtype=torch.int32)
    hole, mover = ~live & (at < total), live & (at >= total)
    # the k-th page behind the end goes to the k-th hole
    holes = torch.argsort((~hole).to(torch.uint8), stable=True).to(torch.int32)
    movers = torch.argsort((~mover).to(torch.uint8), stable=True).to(torch.int32)
    kth = (torch.cumsum(mover.to(torch.int32), 0) - 1).clamp(min=0)
    name = torch.where(mover, holes[kth], torch.where(live, at, torch.full_like(at, -1)))
    s["out_table"].copy_(torch.where(table >= 0, name[table.clamp(min=0).long()], torch.full_like(table, -1)))
    s["out_ref"].zero_()
    s["out_ref"].index_add_(0, name.clamp(min=0).long(), torch.where(live, ref, 0))
    # at most half of the pool can move; slots behind the last mover copy a page onto itself
    most = min(pool - pool // 2, pool)
    move = at[:most] < mover.sum()
    src = torch.where(move, movers[:most], 0)
    dst = torch.where(move, holes[:most], 0)
    keep = [x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in (s["k_cache"], s["v_cache"])]
    for x in keep:
        first = x[:, :1].clone()
        x[:, dst.long()] = x[:, src.long()]
        # page 0 is a hole itself only where the first mover went there
        x[:, :1] = torch.where(hole[0], x[:, movers[:1].long()], first)
    return dict(table=s["out_table"], ref=s["out_ref"], total=total.view(1), k_cache=s["k_cache"], v_cache=s["v_cache"])


# ------------------------------------------------------------ from the definition
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attend":
        return _attend_exact(s)
    if op == "append":
        return _append_exact(s)
    return {"round": _round_exact, "fork": _fork_exact, "compact": _compact_exact}[op](s)


def _attend_exact(s):
    """One request and KV head at a time, over the keys that it has."""
    c = s["case"]
    lens, ell, _ = _lengths(c)
    H, D, page = c["kv_heads"], c["dim"], c["page"]
    group = c["heads"] // H
    if 4 * D * c["heads"] * sum((n + e + 1) * (e + 1) for n, e in zip(lens, ell)) > 2e12:
        return None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    rows, q = out.view(-1, c["heads"], D), s["q"].view(-1, c["heads"], D)
    first = 0
    for b, (n, e) in enumerate(zip(lens, ell)):
        base = first if c["packed"] else b * (c["gamma"] + 1)
        first += e + 1
        at = torch.arange(n + e + 1, device="cuda")
        pages, off = s["table"][b, at // page].long(), at % page
        pos = torch.arange(n, n + e + 1, device="cuda")
        gap = pos[:, None] - at[None, :]
        hidden = gap < 0
        if c["window"]:
            hidden |= (gap >= c["window"]) & (at[None, :] >= c["sinks"])
        for h in range(H):
            K = s["k_cache"][:, :, h].view(torch.uint8)[pages, off].view(s["k_cache"].dtype).double() \
                if c["cache"] == "e4m3" else s["k_cache"][pages, off, h].double()
            V = s["v_cache"][:, :, h].view(torch.uint8)[pages, off].view(s["v_cache"].dtype).double() \
                if c["cache"] == "e4m3" else s["v_cache"][pages, off, h].double()
            if s["k_scale"] is not None:
                K, V = K * s["k_scale"][h].double(), V * s["v_scale"][h].double()
            Q = q[base:base + e + 1, h * group:(h + 1) * group].double()
            x = torch.einsum("rgd,td->rgt", Q, K) / math.sqrt(D)
            x = torch.where(hidden[:, None, :], torch.full_like(x, -math.inf), x)
            rows[base:base + e + 1, h * group:(h + 1) * group] = torch.einsum("rgt,td->rgd", torch.softmax(x, -1), V)
    return out


def _append_exact(s):
    """Complex rotation in 64 bits, and the entries put one request at a time."""
    c = s["case"]
    lens, ell, _ = _lengths(c)
    H, D, page, half = c["kv_heads"], c["dim"], c["page"], c["rotary"] // 2
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    freq = torch.from_numpy(_frequencies(c)).cuda()

    def turned(x, pos):
        x = x.double().clone()
        z = x[..., :2 * half].unflatten(-1, (half, 2)) if c["interleaved"] else \
            x[..., :2 * half].unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(freq), pos.double()[:, None] * freq)[:, None]
        z = torch.view_as_real(z)
        x[..., :2 * half] = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return x

    first = 0
    for b, (n, e) in enumerate(zip(lens, ell)):
        base = first if c["packed"] else b * (c["gamma"] + 1)
        first += e + 1
        pos = torch.arange(n, n + e + 1, device="cuda")
        at = slice(base, base + e + 1)
        out.view(-1, c["heads"], D)[at] = turned(s["q"].view(-1, c["heads"], D)[at], pos)
        new = [turned(s["k"].view(-1, H, D)[at], pos), s["v"].view(-1, H, D)[at].double()]
        pages = s["table"][b, pos // page].long()
        for cache, x, scale in zip(caches, new, (s["k_scale"], s["v_scale"])):
            if scale is not None:
                x = (x / scale.double()[:, None]).clamp(-448.0, 448.0)
            cache[pages, pos % page] = x
    return dict(q=out, k_cache=caches[0], v_cache=caches[1])


def _lists(s):
    return s["table"].tolist(), s["num"].tolist(), s["ref"].tolist(), s["cache_len"].tolist()


def _round_exact(s):
    """The pages by hand, request after request; only the new entries of the plain lists change."""
    c = s["case"]
    table, num, ref, lens = _lists(s)
    _, ell, acc = _lengths(c)
    free = iter([i for i, n in enumerate(ref) if n == 0])
    for b, n in enumerate(lens):
        while num[b] * c["page"] < n + ell[b] + 1:
            table[b][num[b]] = page = next(free)
            ref[page] += 1
            num[b] += 1
    reserved = [list(r) for r in table]
    new_len = [n + a + 1 for n, a in zip(lens, acc)]
    for b, n in enumerate(new_len):
        for slot in range(num[b]):
            first, behind = slot * c["page"], (slot + 1) * c["page"]
            unseen = c["window"] and first >= c["sinks"] and behind <= n - c["window"] + 1
            if table[b][slot] >= 0 and (first >= n or unseen):
                ref[table[b][slot]] -= 1
                table[b][slot] = -1
        num[b] = min(num[b], _pages(n, c["page"]))
    return dict(reserved=_ints(reserved), table=_ints(table), num=_ints(num), ref=_ints(ref), new_len=_ints(new_len),
                status=_ints([0] * c["B"]))


def _fork_exact(s):
    c = s["case"]
    page = c["page"]
    table, num, ref, lens = _lists(s)
    free = iter([i for i, n in enumerate(ref) if n == 0])
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        n = lens[b] = lens[a]
        num[b] = _pages(n, page)
        table[b][:n // page] = table[a][:n // page]
        if n % page:
            table[b][n // page] = new = next(free)
            for x in caches:
                x[:, new, :n % page] = x[:, table[a][n // page], :n % page]
        for slot in range(num[b]):
            ref[table[b][slot]] += 1
    return dict(table=_ints(table), num=_ints(num), ref=_ints(ref), cache_len=_ints(lens), k_cache=caches[0],
                v_cache=caches[1], status=_ints([0] * c["forks"]))


def _compact_exact(s):
    table, num, ref, _ = _lists(s)
    live = [i for i, n in enumerate(ref) if n > 0]
    total = len(live)
    holes = [i for i in range(total) if ref[i] == 0]
    moved = dict(zip([i for i in live if i >= total], holes))
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    for x in caches:
        x[:, list(moved.values())] = x[:, list(moved.keys())]
    out_ref = [0] * len(ref)
    for i in live:
        out_ref[moved.get(i, i)] = ref[i]
    return dict(table=_ints([[moved.get(i, i) for i in r] for r in table]), ref=_ints(out_ref), total=_ints([total]),
                k_cache=caches[0], v_cache=caches[1])
