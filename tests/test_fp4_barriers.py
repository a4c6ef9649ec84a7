"""Waits of the projections' tile kernel as models on the CPU, which take what they model from the kernel's source: nothing
here makes a GPU wait."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "compressed_sparse_attention_07_gb300",
                      "csrc", "fp4_tiles.cu")


def _copying_loops():
    """The source of the two warps that issue copies, in order."""
    text = open(SOURCE).read()
    a, b, c = (text.index(s) for s in ("if (warp == 0) {", "} else if (warp == 1) {", "} else if (warp == 2) {"))
    return text[a:b], text[b:c]


def _lane(runs, steps, gives_up, votes_back):
    """What one lane of a copying warp does, as the names of the whole warp's operations that it takes part in; sent the
    outcome of each vote.  gives_up: the step whose wait runs out for this lane, or None."""
    ok, n = True, 0
    for _ in range(runs):
        if not ok:
            break
        yield "uniform"
        for _ in range(steps):
            if gives_up == n:
                ok = False
            vote = yield "vote", ok
            if votes_back:
                ok = vote
            if not vote:
                break
            yield "elect"
            n += 1
    yield "end"


def _run(runs, steps, give_up, votes_back):
    """Whether all lanes meet in every operation of the warp."""
    lanes = [_lane(runs, steps, g, votes_back) for g in give_up]
    at = [next(lane) for lane in lanes]
    while True:
        names = {a if isinstance(a, str) else a[0] for a in at}
        if len(names) > 1:
            return False  # lanes wait for one another at different places
        if names == {"end"}:
            return True
        outcome = all(a[1] for a in at) if names == {"vote"} else None
        at = [lane.send(outcome) for lane in lanes]


@pytest.mark.parametrize("warp", [0, 1])
def test_lanes_of_a_copying_warp_leave_together(warp):
    """A wait that runs out may do so for some lanes alone: what the vote on it says holds for all of them."""
    code = _copying_loops()[warp]
    assert len(re.findall(r"__all_sync\(", code)) == 1 and len(re.findall(r"\buniform\(", code)) >= 2
    votes_back = re.search(r"\bok = __all_sync\(0xffffffffu, ok\);[^\n]*\s*if \(!ok\) break;", code) is not None
    rnd = random.Random(warp)
    for _ in range(300):
        runs, steps = rnd.randint(1, 3), rnd.randint(1, 4)
        some = rnd.randint(0, 32)
        give_up = [rnd.randrange(runs * steps) if i < some else None for i in range(32)]
        assert _run(runs, steps, give_up, votes_back)


def test_a_vote_that_is_not_taken_back_parts_the_lanes():
    assert not _run(2, 2, [0] * 5 + [None] * 27, False)
    assert _run(2, 2, [None] * 32, False)


ROWS = os.path.join(os.path.dirname(SOURCE), "fp4_rows.cu")


def _ring(units, slots, lost, guarded):
    """A warp of the few-row kernel: units through a ring of bulk copies, of which those in `lost` never land; lane 0's
    waits run out on them.  None, or what went wrong."""
    arrived, landed, ok = [0] * slots, [0] * slots, True  # phases begun and over, of each place

    def fetch(u):
        s = u % slots
        if arrived[s] > landed[s]:
            return False  # an arrival too many, and two copies to one place
        arrived[s] += 1
        if u not in lost:
            landed[s] += 1
        return True

    for u in range(min(units, slots)):
        fetch(u)
    for u in range(units):
        if ok and landed[u % slots] <= u // slots:
            ok = False  # the wait ran out; no more waits
        if u + slots < units and (ok or not guarded) and not fetch(u + slots):
            return "a copy to a place whose copy is on its way"
    return None


def test_no_copy_starts_after_a_wait_that_ran_out():
    text = open(ROWS).read()
    loop = text[text.index("for (int u = u0; u < u1; ++u) {"):]
    guarded = re.search(r"if \(lane == 0 && ok && u \+ slots < u1\)[^;]*fetch\(\)", loop) is not None
    rnd = random.Random(1)
    for _ in range(500):
        units, slots = rnd.randint(1, 40), rnd.randint(2, 8)
        assert _ring(units, slots, {rnd.randrange(units)} if rnd.random() < 0.8 else set(), guarded) is None


def test_copies_after_a_wait_that_ran_out_are_found_wrong():
    assert _ring(9, 3, {2}, False) and _ring(9, 3, set(), False) is None
