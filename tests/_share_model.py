"""Plain models of the calls for batches that share prefixes: a plan's groups as
lists, and attention cases whose page tables begin with the same pages."""
from __future__ import annotations

import torch

from tests._cache_model import Case


def groups(table, lens, page, least, passes=32):
    """(leader, shared) of each request, by the definition of spec_share_plan;
    lens: -1 of a request that has an error."""
    B = len(table)
    full = [n // page if n >= 0 else 0 for n in lens]
    leader, shared = list(range(B)), [0] * B
    left = [b for b in range(B) if full[b] > 0 and table[b][0] >= 0]
    for _ in range(passes):
        rest = []
        for first in sorted({table[b][0] for b in left}):
            members = [b for b in left if table[b][0] == first]
            head = members[0]
            depth = {}
            for b in members[1:]:
                d = 0
                while d < min(full[b], full[head]) and table[b][d] == table[head][d] and table[b][d] >= 0:
                    d += 1
                depth[b] = d
            best = max([(d * sum(x >= d for x in depth.values()), sum(x >= d for x in depth.values()), d)
                        for d in depth.values() if d * page >= least], default=(0, 0, 0))
            d = best[2]
            for b in members:
                if d and (b == head or depth[b] >= d):
                    leader[b], shared[b] = head, d
                elif b != head:
                    rest.append(b)
        left = sorted(rest)
    return leader, shared


class SharedCase(Case):
    """A Case in which the requests of each (members, pages) of `share` have the
    first of them's leading pages."""

    def __init__(self, *, share, least=1, **kw):
        super().__init__(**kw)
        self.least = least
        for members, pages in share:
            assert all(self.lens[b] >= pages * self.page for b in members)
            self.table[members, :pages] = self.table[members[0], :pages].clone()

    def model(self):
        return groups(self.table.tolist(), self.lens, self.page, self.least)

    def make_plan(self, sv, lens=None, ell=None, **kw):
        """lens, ell: others than the case's."""
        i32 = torch.int32
        packed = self.row is not None
        return sv.share_plan(self.to(self.table), self.to(torch.tensor(self.lens if lens is None else lens, dtype=i32)),
                             self.to(torch.tensor(self.ell if ell is None else ell, dtype=i32)), self.to(self.row),
                             gamma=self.gamma, page_size=self.page, rows=self.q.shape[0] if packed else None,
                             least=self.least, **kw)

    def call(self, sv, q=None, caches=None, plan=None, table=None, **kw):
        caches = caches or self.caches()
        plan = self.make_plan(sv)[0] if plan is None else plan
        return sv.attend_shared(self.to(self.q) if q is None else q, caches[0], caches[1],
                                self.to(self.table if table is None else table), plan, gamma=self.gamma,
                                k_scale=self.to(self.k_scale), v_scale=self.to(self.v_scale), **kw)


class Banded:
    """Buffers of a size between bands of a known byte."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype, fill=None):
        n = int(torch.tensor(shape).prod()) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((n + 2 * 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        x = raw[4096:4096 + n].view(dtype).view(shape)
        if fill is not None:
            x.fill_(fill)
        self.all.append((raw, n))
        return x

    def check(self):
        torch.cuda.synchronize()
        for raw, n in self.all:
            assert (raw[:4096] == 0xA5).all() and (raw[4096 + n:] == 0xA5).all()
