"""Plain models of the key-value cache calls for the tests: attention and
rotary positions in 64 bits, pages as Python lists."""
from __future__ import annotations

import math

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


class Case:
    """Inputs of an attend call on `device`, made on the CPU from a seed."""

    def __init__(self, *, lens, ell, gamma, heads=8, kv_heads=2, dim=64, page=16, dtype="bf16", cache="bf16",
                 window=0, sinks=0, packed=False, layout="tokens", seed=0, spread=2.0, device="cuda", poison=True):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.lens, self.ell, self.gamma, self.page = lens, ell, gamma, page
        self.heads, self.kv_heads, self.dim, self.window, self.sinks = heads, kv_heads, dim, window, sinks
        self.dtype, self.cache = dtype, cache
        need = [-(-(n + e + 1) // page) for n, e in zip(lens, ell)]
        slots, pool = max(need) + 1, sum(need) + 5
        perm = torch.randperm(pool, generator=g).tolist()
        table = torch.full((B, slots), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            for s in range(n):
                table[b, s] = perm.pop()
        self.table = table
        dt, ct = TYPES[dtype], TYPES[cache]

        def values(shape, std, t):
            return (torch.randn(shape, generator=g) * std).to(t)

        std = 20.0 if cache == "e4m3" else 1.0
        self.k = values((pool, page, kv_heads, dim), std, ct)
        self.v = values((pool, page, kv_heads, dim), std, ct)
        self.k_scale = self.v_scale = None
        if cache == "e4m3":
            self.k_scale = torch.rand(kv_heads, generator=g) * 0.05 + 0.02
            self.v_scale = torch.rand(kv_heads, generator=g) * 0.05 + 0.02
        if poison:  # what no row sees holds NaN, and pages behind the window are gone
            seen = torch.zeros(pool, page, dtype=torch.bool)
            for b in range(B):
                for t in range(lens[b] + ell[b] + 1):
                    if self.any_sees(b, t):
                        seen[table[b, t // page], t % page] = True
            for x in (self.k, self.v):
                raw = x.float()
                raw[~seen] = float("nan")
                x.copy_(raw.to(ct))
            for b in range(B):
                for s in range(need[b]):
                    if not seen[table[b, s]].any():
                        table[b, s] = -1
        n = [e + 1 for e in ell]
        self.row = torch.tensor(np.cumsum(n) - n, dtype=torch.int32) if packed else None
        rows = (sum(n),) if packed else (B, gamma + 1)
        self.q = values(rows + (heads, dim), spread, dt)
        self.layout = layout
        self.device = device

    def any_sees(self, b, t):
        return any(self.sees(self.lens[b] + j, t) for j in range(self.ell[b] + 1))

    def sees(self, p, t):
        return t <= p and (self.window == 0 or p - t < self.window or t < self.sinks)

    def base(self, b):
        return int(self.row[b]) if self.row is not None else b * (self.gamma + 1)

    def to(self, x):
        return None if x is None else x.to(self.device)

    def caches(self):
        """The caches on the device in the case's layout."""
        out = []
        for x in (self.k, self.v):
            x = x.to(self.device)
            if self.layout == "heads":      # [pages, heads, page, dim] in memory
                x = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
            elif self.layout == "pair":     # K and V of a page side by side, as slices
                x = torch.stack([x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x] * 2, 1)
                x = (x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x)[:, 1]
            out.append(x)
        return out

    def call(self, sv, q=None, caches=None, **kw):
        caches = caches or self.caches()
        return sv.attend(self.to(self.q) if q is None else q, caches[0], caches[1], self.to(self.table),
                         self.to(torch.tensor(self.lens, dtype=torch.int32)),
                         self.to(torch.tensor(self.ell, dtype=torch.int32)), self.to(self.row), gamma=self.gamma,
                         window=self.window, sinks=self.sinks, k_scale=self.to(self.k_scale),
                         v_scale=self.to(self.v_scale), **kw)

    def expect(self, scale=None):
        """(out, lse, tolerance) in 64 bits, of the rows that exist (others NaN,
        tolerance 0)."""
        scale = self.dim ** -0.5 if scale is None else scale
        D, group = self.dim, self.heads // self.kv_heads
        rows = self.q.reshape(-1, self.heads, D)
        out = torch.full(rows.shape, float("nan"), dtype=torch.float64)
        tol = torch.zeros(rows.shape, dtype=torch.float64)
        lse = torch.full(rows.shape[:2], float("nan"), dtype=torch.float64)
        eps = torch.finfo(TYPES[self.dtype]).eps
        # weights are rounded to the type of the product with v: 16-bit rows' own,
        # fp16 under an e4m3 cache, 32 bits for fp32 rows
        weight = torch.finfo(torch.float16).eps if self.cache == "e4m3" else eps
        small = 2.0 ** -25 if self.dtype == "fp16" or self.cache == "e4m3" else 0.0  # fp16: half the least step
        for b in range(len(self.lens)):
            n, e = self.lens[b], self.ell[b]
            for j in range(e + 1):
                p = n + j
                t = torch.tensor([t for t in range(p + 1) if self.sees(p, t)])
                pages = self.table[b][t // self.page].long()
                for h in range(self.kv_heads):
                    K = self.k[:, :, h].float()[pages, t % self.page].double()
                    V = self.v[:, :, h].float()[pages, t % self.page].double()
                    if self.k_scale is not None:
                        K, V = K * self.k_scale[h].double(), V * self.v_scale[h].double()
                    hs = slice(h * group, (h + 1) * group)
                    Q = rows[self.base(b) + j, hs].double()
                    s = Q @ K.T * scale
                    m = s.amax(-1, keepdim=True)
                    w = torch.exp(s - m)
                    l = w.sum(-1, keepdim=True)
                    o = w / l @ V
                    # fp32 score: D products and sums of 2^-24 each, at most, and a
                    # bf16 query under an e4m3 cache passes through fp16 (scaled)
                    off = (D + 8) * 2.0 ** -24 * ((Q.abs() @ K.abs().T) * abs(scale)).amax(-1, keepdim=True)
                    A = w / l @ V.abs()
                    # twice the score's error in a weight over its sum, exp2 and sums in fp32
                    r = weight / 2 + 2 * off + 2.0 ** -20 + (len(t) + 64) * 2.0 ** -24
                    tiny = small * (1.0 + V.abs().sum(0) / l)
                    out[self.base(b) + j, hs] = o
                    tol[self.base(b) + j, hs] = eps / 2 * o.abs() * 1.01 + r * A + tiny
                    lse[self.base(b) + j, hs] = (m + torch.log(l))[:, 0]
        shape = self.q.shape
        return out.view(shape), lse.view(shape[:-1]), tol.view(shape)

    def check(self, got, lse=None, **kw):
        out, want_lse, tol = self.expect(**kw)
        have = ~torch.isnan(out)
        got = got.float().double().cpu()
        assert torch.isfinite(got[have]).all()
        over = ((got - out).abs() - tol)[have]
        assert (over <= 0).all(), (float(over.max()), float((got - out).abs()[have].max()))
        if lse is not None:
            have = ~torch.isnan(want_lse)
            d = (lse.double().cpu() - want_lse)[have].abs()
            assert (d <= 2e-5 * (1 + want_lse[have].abs())).all(), float(d.max())


def rotated(x, pos, freq, interleaved, mscale=1.0):
    """x [heads, dim] float64 turned to position pos."""
    x = np.array(x, dtype=np.float64)
    half = len(freq)
    a = pos * np.asarray(freq, np.float64)
    c, s = np.cos(a) * mscale, np.sin(a) * mscale
    i, j = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    u, v = x[:, i].copy(), x[:, j].copy()
    x[:, i], x[:, j] = u * c - v * s, u * s + v * c
    return x


class Pool:
    """Pages as lists, by the definitions of the calls."""

    def __init__(self, B, slots, pages, page):
        self.B, self.slots, self.pages, self.page = B, slots, pages, page
        self.table = [[-1] * slots for _ in range(B)]
        self.num, self.len, self.ref = [0] * B, [0] * B, [0] * pages

    def tensors(self, device="cuda"):
        def i32(x):
            return torch.tensor(x, dtype=torch.int32, device=device)
        return i32(self.table), i32(self.num), i32(self.ref), i32(self.len)

    def same(self, table, num, ref, length):
        assert table.cpu().tolist() == self.table
        assert num.cpu().tolist() == self.num
        assert ref.cpu().tolist() == self.ref
        assert length.cpu().tolist() == self.len

    def free(self):
        return [i for i, n in enumerate(self.ref) if n == 0]

    def reserve(self, ell, gamma):
        status, free, out = [], self.free(), False
        for b in range(self.B):
            need = -(-(self.len[b] + ell[b] + 1) // self.page)
            if not 0 <= ell[b] <= gamma:
                status.append(-5)
            elif need > self.slots or self.len[b] < 0:
                status.append(-16)
            elif need <= self.num[b]:
                status.append(0)
            elif out or need - self.num[b] > len(free):
                out = True
                status.append(-15)
            else:
                for s in range(self.num[b], need):
                    self.table[b][s] = free.pop(0)
                    self.ref[self.table[b][s]] = 1
                self.num[b] = need
                status.append(0)
        return status

    def drop(self, b, s):
        if self.table[b][s] >= 0:
            self.ref[self.table[b][s]] -= 1
        self.table[b][s] = -1

    def commit(self, accept, window=0, sinks=0):
        for b in range(self.B):
            now = self.len[b] + accept[b] + 1
            if accept[b] < -1 or now > self.num[b] * self.page:
                continue
            keep = -(-now // self.page)
            for s in range(self.num[b]):
                # the next token, at position `now`, sees t > now - window
                unseen = window and all(t >= sinks and now - t >= window
                                        for t in range(s * self.page, (s + 1) * self.page))
                if s >= keep or unseen:
                    self.drop(b, s)
            self.num[b], self.len[b] = keep, now

    def end(self, requests):
        for b in requests:
            if 0 <= b < self.B:
                for s in range(self.num[b]):
                    self.drop(b, s)
                self.num[b] = self.len[b] = 0

    def fork(self, src, dst):
        """Status of each, and [(page, copy, tokens)]."""
        status, copies, ok = [], [], []
        for s, d in zip(src, dst):
            if not (0 <= s < self.B and 0 <= d < self.B) or dst.count(d) > 1 or d in src:
                status.append(-18)
            elif self.len[s] < 0 or -(-self.len[s] // self.page) > self.num[s]:
                status.append(-16)
            elif self.len[s] % self.page and not 0 <= self.table[s][self.len[s] // self.page] < self.pages:
                status.append(-17)
            else:
                status.append(0)
        for i, d in enumerate(dst):
            if status[i] == 0:
                self.end([d])
        free = self.free()
        for i, (s, d) in enumerate(zip(src, dst)):
            if status[i]:
                continue
            whole, tail = divmod(self.len[s], self.page)
            if tail and not free:
                status[i] = -15
                continue
            self.table[d][:whole] = self.table[s][:whole]
            for p in self.table[s][:whole]:
                if p >= 0:
                    self.ref[p] += 1
            if tail:
                self.table[d][whole] = p = free.pop(0)
                self.ref[p] = 1
                copies.append((self.table[s][whole], p, tail))
            self.num[d], self.len[d] = whole + (tail > 0), self.len[s]
        return status, copies

    def compact(self):
        """[(from, to)] of the moved pages."""
        live = [i for i, n in enumerate(self.ref) if n > 0]
        N = len(live)
        moves = list(zip([i for i in live if i >= N], [i for i in range(N) if self.ref[i] == 0]))
        name = dict(moves)
        ref = [0] * self.pages
        for i in live:
            ref[name.get(i, i)] = self.ref[i]
        self.ref = ref
        self.table = [[name.get(p, p) for p in r] for r in self.table]
        return N, moves


def need_pages(n, page):
    return math.ceil(n / page)
