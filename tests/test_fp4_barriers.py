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
    a, b, c = (text.index("auto %s = " % s) for s in ("copy_weights", "copy_rows", "products"))
    return text[a:b], text[b:c]


def _lane(runs, steps, gives_up, votes_back):
    """What one lane of a copying warp does, as the names of the whole warp's operations that it takes part in; sent the
    outcome of each vote.  gives_up: the step whose wait runs out for this lane, or None.  votes_back: whether lanes take
    the outcome of a vote for their own behind a run's steps."""
    ok, n = True, 0
    for _ in range(runs):
        if not ok:
            break
        yield "uniform"
        for _ in range(steps):
            if gives_up == n:
                ok = False
            vote = yield "vote", ok
            if not vote:
                break
            yield "elect"
            n += 1
        if votes_back:
            ok = yield "vote", ok
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
    assert len(re.findall(r"\bif \(!__all_sync\(0xffffffffu, ok\)\) break;", code)) == 1
    assert len(re.findall(r"\buniform\(", code)) >= 2 and re.search(r"i < runs && ok;", code)
    # the vote behind the steps: after the loop over them has closed
    votes_back = re.search(r"__syncwarp\(\);\s*\}\s*ok = __all_sync\(0xffffffffu, ok\);", code) is not None
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


# ---- the tile kernel's barriers under random schedules (Barrier, _wait and _check as for kv_tiles_kernel) ----

from tests.test_kv_barriers import Barrier, Wrong, _check, _wait  # noqa: E402


def _value(expr, env):
    """A C expression of numbers, names, comparisons, + - * / and conditionals."""
    at, depth = None, 0
    for i, ch in enumerate(expr):
        depth += (ch == "(") - (ch == ")")
        if ch == "?" and depth == 0:
            at = i
            break
    if at is None:
        expr = re.sub(r"&&", " and ", re.sub(r"\|\|", " or ", expr))
        return eval(expr.replace("/", "//").replace("true", "True").replace("false", "False"), {}, env)  # noqa: S307
    nest = depth = 0
    for i in range(at + 1, len(expr)):
        depth += (expr[i] == "(") - (expr[i] == ")")
        if depth == 0:
            nest += (expr[i] == "?") - (expr[i] == ":")
            if nest < 0:
                return _value(expr[at + 1:i] if _value(expr[:at], env) else expr[i + 1:], env)
    raise ValueError(expr)


def _rings(tok, apart):
    text = open(SOURCE).read()
    text = text[text.index("struct Rings {"):]
    text = text[:text.index("static_assert")]
    env = dict(kTok=tok, kApart=apart, kTileRows=128, kTileBytes=9216)
    for decl in re.findall(r"static constexpr (?:int|bool) ([^;]*);", text):
        for name, expr in re.findall(r"(\w+) = ((?:[^,()]|\([^()]*\))+)", decl):
            try:
                env[name] = _value(expr.strip(), env)
            except NameError:
                pass  # (not a size of a ring)
    return env


class Tiles:
    """Runs of so many steps through a CTA.  Steps are numbered through all runs; a place holds the number of the step that
    was last written there."""

    def __init__(self, seed, runs, r):
        self.rnd, self.runs, self.r = random.Random(seed), runs, r
        self.steps = sum(runs)
        self.full_p, self.empty_p = [Barrier(1) for _ in range(r["kP"])], [Barrier(4) for _ in range(r["kP"])]
        joint = r["kJoint"]
        self.full_x, self.empty_x = [Barrier(1) for _ in range(r["kX"])], [Barrier(1) for _ in range(r["kX"])]
        self.full_a, self.empty_a = [Barrier(5 if joint else 4) for _ in range(r["kS"])], [Barrier(1) for _ in range(r["kS"])]
        if joint:  # the same barriers, of a step
            self.full_x, self.empty_x = self.full_a, self.empty_a
        self.full_d, self.empty_d = [Barrier(1) for _ in range(r["kD"])], [Barrier(4) for _ in range(r["kD"])]
        self.p, self.x = [None] * r["kP"], [None] * r["kX"]
        self.a = {}
        self.d = [None] * r["kD"]          # (run, steps summed) of each accumulator
        self.flying, self.issued, self.out = [], [], {w: [] for w in range(4)}

    def spans(self):
        for run, steps in enumerate(self.runs):
            for first in range(0, steps, self.r["kSpan"]):
                yield run, min(steps - first, self.r["kSpan"])

    def weights(self):
        k = self.r["kP"]
        for n in range(self.steps):
            if n >= k:
                yield from _wait(self.empty_p[n % k], n // k - 1)
            self.p[n % k] = None

            def land(n=n):
                self.p[n % k] = n
                self.full_p[n % k].arrive()
            self.flying.append(land)
            yield

    def rows(self):
        k, per = self.r["kX"], 2 // self.r["kBoxes"]
        for n in range(self.steps * per):
            if n >= k:
                yield from _wait(self.empty_x[n % k], n // k - 1)
            self.x[n % k] = None

            def land(n=n):
                self.x[n % k] = n
                self.full_x[n % k].arrive()
            self.flying.append(land)
            yield

    def decode(self, group, w):
        kp, ks = self.r["kP"], self.r["kS"]
        for n in range(group, self.steps, self.r["kSets"]):
            yield from _wait(self.full_p[n % kp], n // kp)
            _check(self.p[n % kp] == n, "weights of another step")
            yield
            _check(self.p[n % kp] == n, "weights overwritten while they were read")
            self.empty_p[n % kp].arrive()
            if n >= ks:
                yield from _wait(self.empty_a[n % ks], n // ks - 1)
            self.a[w, n % ks] = n
            yield
            self.full_a[n % ks].arrive()

    def issue(self):
        r, n, box = self.r, 0, 0
        for at, (run, steps) in enumerate(self.spans()):
            s = at % r["kD"]
            if at >= r["kD"]:
                yield from _wait(self.empty_d[s], at // r["kD"] - 1)
            for i in range(steps):
                yield from _wait(self.full_a[n % r["kS"]], n // r["kS"])
                for _ in range(2 // r["kBoxes"]):
                    if not r["kJoint"]:
                        yield from _wait(self.full_x[box % r["kX"]], box // r["kX"])

                    def run_products(n=n, box=box, s=s, first=i == 0, run=run):
                        _check(all(self.a.get((w, n % r["kS"])) == n for w in range(4)), "products of other weights")
                        _check(self.x[box % r["kX"]] == box, "products of other rows")
                        if box % (2 // r["kBoxes"]) == 0:
                            self.d[s] = (run, 1) if first else (run, self.d[s][1] + 1)
                    self.issued.append(run_products)
                    if not r["kJoint"]:
                        self.issued.append(self.empty_x[box % r["kX"]].arrive)
                    box += 1
                self.issued.append(self.empty_a[n % r["kS"]].arrive)
                n += 1
                yield
            self.issued.append(self.full_d[s].arrive)
            yield

    def store(self, w):
        for at, (run, steps) in enumerate(self.spans()):
            s = at % self.r["kD"]
            yield from _wait(self.full_d[s], at // self.r["kD"])
            _check(self.d[s] == (run, steps), "sums of something else")
            yield
            _check(self.d[s] == (run, steps), "sums overwritten while they were read")
            self.out[w].append((run, steps))
            self.empty_d[s].arrive()
            yield

    def run(self):
        warps = [self.weights(), self.rows(), self.issue()] + [self.store(w) for w in range(4)]
        warps += [self.decode(g, w) for g in range(self.r["kSets"]) for w in range(4)]
        weight = [self.rnd.choice((1, 1, 3, 10)) for _ in warps]
        for _ in range(400000):
            if self.flying and self.rnd.random() < 0.3:
                self.flying.pop(self.rnd.randrange(len(self.flying)))()
            if self.issued and self.rnd.random() < 0.5:
                self.issued.pop(0)()
            k = self.rnd.choices(range(len(warps)), weight)[0]
            try:
                next(warps[k])
            except StopIteration:
                del warps[k], weight[k]
                if not warps:
                    for out in self.out.values():
                        for run, steps in enumerate(self.runs):
                            _check(sum(n for r, n in out if r == run) == steps, "steps that were not summed")
                    return
        raise Wrong("a standstill")


@pytest.mark.parametrize("tok,apart", [(t, False) for t in (16, 32, 64, 128, 256)] + [(t, True) for t in (16, 32, 64, 128)])
def test_no_schedule_of_the_tiles_goes_wrong(tok, apart):
    r = _rings(tok, apart)
    assert r["kSpan"] % 2 == 0 and r["kP"] % r["kSets"] == 0 and (not r["kJoint"] or r["kX"] == r["kS"])
    for seed in range(25):
        rnd = random.Random(seed)
        runs = [rnd.choice((1, 2, 3, 5, 9, 14)) for _ in range(rnd.randint(1, 4))]
        Tiles(seed, runs, r).run()


@pytest.mark.parametrize("wrong", [dict(kP=3, kSets=2), dict(kS=2, kX=2, kSets=4)])
def test_rings_that_do_not_fit_their_sets_are_found_wrong(wrong):
    r = dict(_rings(64, True), **wrong)
    failures = 0
    for seed in range(25):
        try:
            Tiles(seed, [14, 9], r).run()
        except Wrong:
            failures += 1
    assert failures
