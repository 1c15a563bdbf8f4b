"""The waits of the tensor-core attention kernel, on the CPU.

A wait on an mbarrier's parity passes when the awaited phase is over, and also
while the barrier is two phases behind it.  The model runs the products in their
order of issue against the two softmax streams, in every interleaving: each
product, copy and warp may be late by any amount.  What a unit's end waits for
is read from the kernel's source."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_softmax_gb300", "csrc")


def source():
    with open(os.path.join(CSRC, "specv_attend_tc.cuh")) as f:
        return f.read()


def unit_end():
    """The barrier that the softmax warps wait for before they read a unit's
    output, and whether one product stream's or a unit's phases pass on it."""
    text = source()
    upto = text.index("s_ml[0][row] = m;")
    name, place = re.findall(r"tc_wait\(&(\w+)(\[s\])?, ", text[:upto])[-1]
    products = text[text.index("for (int i = 0; i < w.nt + NB; ++i)"):]
    loop = products[:products.index("first += w.nt;")]
    behind = loop.rstrip().endswith("tc_commit(one, &%s);" % name)   # behind a unit's last product
    assert bool(place) != behind
    return "stream" if place else "unit"


def passes(done, phase):
    """A parity wait for phase `phase` of a barrier with `done` phases over: it
    sees the parity of the phase under way, and nothing else."""
    return (done - phase) % 2 == 1


def early_reads(units, ahead, end):
    """Every interleaving of the products and the two streams over `units` (tiles
    each); the set of what was read before it was there, and of ends that are none."""
    start = [sum(units[:u]) for u in range(len(units))]
    # products in order of issue: ("S" or "O", unit, tile), ("U", unit): the unit's commit
    issue = []
    for u, nt in enumerate(units):
        for i in range(nt + ahead):
            if i >= ahead:
                issue.append(("O", u, i - ahead))
            if i < nt:
                issue.append(("S", u, i))
        issue.append(("U", u, 0))
    number = {x: i for i, x in enumerate(issue)}
    # a stream's steps; "fix" is the scaling of the output, which may be left out
    steps = [[], []]
    for s in (0, 1):
        seen = 0
        for u, nt in enumerate(units):
            for t in range(s, nt, 2):
                steps[s].append(("scores", u, t, seen))
                if t >= 2:
                    steps[s].append(("fix", u, t, seen))
                steps[s].append(("weights", u, t, seen))
                seen += 1
            steps[s].append(("end", u, nt, seen))
            steps[s].append(("meet", u, nt, seen))
    weights = {(x[1], x[2]): (s, i) for s in (0, 1) for i, x in enumerate(steps[s]) if x[0] == "weights"}

    bad, known, work = set(), set(), [(0, 0, 0, 0)]

    def over(kind, s, done):
        return sum(1 for x in issue[:done] if x[0] == kind and (s is None or x[2] % 2 == s))

    def of_place(kind, place, done):
        return sum(1 for x in issue[:done] if x[0] == kind and (start[x[1]] + x[2]) % ahead == place)

    while work:
        state = work.pop()
        if state in known:
            continue
        known.add(state)
        issued, done, at = state[0], state[1], state[2:]
        before = len(work)
        if done < issued:
            work.append((issued, done + 1) + at)
        if issued < len(issue):
            kind, u, t = issue[issued]
            go = True
            if kind == "O":
                s, i = weights[u, t]
                g = start[u] + t
                handed = sum(1 for (u2, t2), (s2, i2) in weights.items()
                             if at[s2] > i2 and (start[u2] + t2) % ahead == g % ahead)
                go = passes(handed, g // ahead)
                if go and at[s] <= i:
                    bad.add(("weights", u, t))
            if go:
                work.append((issued + 1, done) + at)
        for s in (0, 1):
            if at[s] == len(steps[s]):
                continue
            what, u, t, seen = steps[s][at[s]]
            go, skip = True, False
            if what == "scores":
                g = start[u] + t
                go = passes(of_place("S", g % ahead, done), g // ahead)
                if go and number["S", u, t] >= done:
                    bad.add(("scores", u, t))
            elif what == "fix":
                skip = True
                go = passes(over("O", s, done), seen - 1)
                if go and number["O", u, t - 2] >= done:
                    bad.add(("fix", u, t))
            elif what == "end":
                if end == "unit":
                    go = passes(over("U", None, done), u)
                elif s < t:
                    go = passes(over("O", s, done), seen - 1)
                if go and any(number["O", u, x] >= done for x in range(s, t, 2)):
                    bad.add(("end", u, s))
            elif what == "meet":
                go = at[1 - s] >= next(i for i, x in enumerate(steps[1 - s]) if x[:2] == ("meet", u))
            if go or skip:
                work.append((issued, done) + tuple(a + (q == s) for q, a in enumerate(at)))
        if len(work) == before and (done < len(issue) or any(at[s] < len(steps[s]) for s in (0, 1))):
            bad.add(("stuck",) + state)
    return bad


UNITS = [(1,), (2,), (3,), (4,), (5,), (6,), (7,), (1, 4), (4, 1), (3, 5), (5, 2, 3), (1, 1, 3), (2, 6)]


@pytest.mark.parametrize("units", UNITS)
@pytest.mark.parametrize("ahead", [2, 3])
def test_no_output_is_read_before_its_products_are_over(units, ahead):
    assert re.search(r"kAhead = D == 64 \? 3 : 2;", source())
    assert early_reads(units, ahead, unit_end()) == set()


def test_the_model_finds_early_reads():
    """A stream's own last phase is not enough where its last scores do not imply
    the product before."""
    assert ("end", 0, 0) in early_reads((3,), 3, "stream")
    assert early_reads((5,), 2, "stream") == set()
    assert early_reads((2,), 3, "stream") == set()


def test_repaired_values_are_told_before_the_tile_is_handed_on():
    """What was taken out of a V tile has to be known to the softmax warps: each
    warp of a team says so before the team's barrier, behind which one thread
    hands the tile on."""
    text = source()
    loop = text[text.index("for (int i = 0; i < 2 * w.nt; ++i, ++item)"):]
    loop = loop[:loop.index("mbar_arrive(&full[slot])")]
    steps = re.findall(r"repair<|s_flags\[u % kTcUnits\], 2\)|meet\(\);", loop)
    assert steps == ["repair<", "s_flags[u % kTcUnits], 2)", "meet();"] * 2


def test_missing_pages_are_told_before_the_tile_is_handed_on():
    """The lanes of a loading warp that find no page say so before lane 0 arrives
    for the tile; votes among them order no memory."""
    text = source()
    loop = text[text.index("s_flags[w.u % kTcUnits], 1)"):]
    loop = loop[:loop.index("mbar_arrive_expect_tx(bar")]
    assert loop.count("__syncwarp();") == 1


def test_after_a_wait_has_run_out_no_slot_is_loaded():
    """A role whose wait has run out goes on without waiting, and gives slots back
    whose copies may be under way.  A loader that took one would arrive on the
    barrier of that copy once too often; so would one that skipped a slot and met
    it again, two phases behind."""
    text = source()
    # loaders: one word for all later slots; over a 16-bit cache the products free them
    assert "uint64_t* freed = F8 ? &raw_empty[slot] : &empty[slot];" in text
    assert re.search(r"ok = ok && __all_sync\(0xffffffffu, \(item < NR \|\| tc_wait\(freed, .*, fail\)\) &&\s+"
                     r"\(F8 \|\| !\*fail\)\);", text)
    assert "if (lane == 0 && ok) mbar_arrive_expect_tx(" in text and "have = have && ok;" in text
    # wideners give back what came by TMA, the repair hands on what did
    assert "ok = tc_wait(&raw_full[rs], (item / NR) & 1, fail) && ok;" in text
    assert re.findall(r"if \((.*)\) mbar_arrive\(&raw_empty\[rs\]\);", text) == ["lt == 0 && ok"]
    assert re.findall(r"if \((.*)\) mbar_arrive\(&full\[slot\]\);", text) == ["lt == 0 && (F8 || !*fail)"]
