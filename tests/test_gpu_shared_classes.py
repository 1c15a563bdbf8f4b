"""Plans of batches with many groups, or many requests that share with nobody,
behind the same first pages: no group is lost, in whatever order they stand."""
import random

import pytest
import torch

from tests._share_model import SharedCase, groups

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


def check(sv, table, lens, page, least):
    slots = max(map(len, table))
    table = [t + [-1] * (slots - len(t)) for t in table]
    t, n = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (table, lens))
    plan, leader, shared = sv.share_plan(t, n, gamma=2, page_size=page, least=least)
    assert sv.read_status(plan) == 0
    want = groups(table, lens, page, least, passes=len(table))
    assert leader.tolist() == want[0]
    assert shared.tolist() == want[1]
    return want


class Pages:
    """Ids by name."""

    def __init__(self):
        self.ids = {}

    def __call__(self, *names):
        return [self.ids.setdefault(n, len(self.ids)) for n in names]

    def run(self, name, n):
        return self(*[(name, i) for i in range(n)])


@pytest.mark.parametrize("lone", [31, 32, 40, 300])
def test_lone_requests_ahead_of_a_group(sv, lone):
    """A common first page, `lone` requests with nothing else in common, and 64 that share 41 pages."""
    p = Pages()
    first = p("system")
    table = [first + p.run(("own", b), 45) for b in range(lone)]
    table += [first + p.run("document", 40) + p.run(("own", lone + b), 5) for b in range(64)]
    leader, shared = check(sv, table, [46 * 16 - 9] * len(table), 16, 256)
    assert leader[lone:] == [lone] * 64 and shared[lone:] == [41] * 64 and not any(shared[:lone])


@pytest.mark.parametrize("chats,samples", [(64, 4), (200, 2), (1000, 4)])
@pytest.mark.parametrize("system", [1, 10, 15])
def test_samples_of_many_chats(sv, chats, samples, system):
    """Samples of each of many chats behind a system prompt that is too short to share."""
    p = Pages()
    common = p.run("system", system)
    order = [c for c in range(chats) for _ in range(samples)]
    random.Random(chats).shuffle(order)
    table = [common + p.run(("chat", c), 30) + p(("own", b)) for b, c in enumerate(order)]
    _, shared = check(sv, table, [(system + 30) * 16 + 5] * len(table), 16, 256)
    assert shared == [system + 30] * len(table)


def test_many_deep_groups_behind_a_long_prompt(sv):
    """A system prompt that is long enough, but each chat's samples save more by their own."""
    p = Pages()
    common = p.run("system", 16)
    order = [c for c in range(40) for _ in range(4)]
    random.Random(1).shuffle(order)
    table = [common + p.run(("chat", c), 900) + p(("own", b)) for b, c in enumerate(order)]
    _, shared = check(sv, table, [916 * 16] * len(table), 16, 256)
    assert shared == [916] * len(table)


@pytest.mark.parametrize("least", [0, 1, 16, 17, 32, 33, 100, 1 << 30])
def test_same_pages_behind_other_ones(sv, least):
    """Rows that are alike at some places only, missing entries among them, and lengths down to zero."""
    for seed in range(6):
        r = random.Random(seed * 100 + least)
        B = r.choice([3, 40, 150])
        few = r.choice([2, 3, 6])
        table = [[r.choice([-1, 0, 1, 2][:few]) if r.random() < 0.5 else 7 + s for s in range(12)] for _ in range(B)]
        for b in range(B):
            if r.random() < 0.4:
                table[b][:r.randint(1, 12)] = table[r.randrange(B)][:r.randint(1, 12)]
                table[b] = (table[b] + [3] * 12)[:12]
        check(sv, table, [r.choice([0, 15, 16, 12 * 16 - 3, r.randint(0, 12 * 16 - 3)]) for _ in range(B)], 16, least)


@pytest.mark.parametrize("B", [34, 300, 1300])
def test_one_page_alike_behind_other_ones(sv, B):
    """All have the page in which a prefix ends, but only some have those before it too."""
    p = Pages()
    r = random.Random(B)
    same = p("page")
    who = [r.randrange(5) if r.random() < 0.2 else ("own", b) for b in range(B)]
    table = [p.run(("first", w), 15) + same + p.run(("own", b), 2) for b, w in enumerate(who)]
    _, shared = check(sv, table, [18 * 16 - 5] * B, 16, 256)
    assert not all(shared) and (any(shared) or B == 34)    # by chance none of the 34


def test_attention_of_many_groups(sv):
    """Fifty pairs, forty lone requests ahead of them, one first page: the rows' values by such a plan."""
    lens = [70 + b % 5 for b in range(140)]
    case = SharedCase(share=[([40 + 2 * i, 41 + 2 * i], 4) for i in range(50)], lens=lens, ell=[b % 3 for b in range(140)],
                      gamma=2, heads=4, kv_heads=2, dim=64, least=48, seed=2)
    case.table[:, 0] = case.table[0, 0]
    plan, leader, shared = case.make_plan(sv)
    assert leader.tolist() == list(range(40)) + [40 + b // 2 * 2 for b in range(100)]
    assert shared.tolist() == [0] * 40 + [4] * 100
    out, ws = case.call(sv, plan=plan)
    assert sv.read_status(ws) == sv.read_status(plan) == 0
    case.check(out)
