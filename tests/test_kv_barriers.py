"""The barriers of kv_tiles_kernel as a model run under random schedules: warps that wait for the parity of a phase, bulk
copies that land at any time, products that run in the order of their issue.  The model has no data but the numbers of
the tiles, and finds a wait that passes on an earlier phase, a tile read before it has landed or overwritten while it is
read, an arrival too many, and a standstill.  The rings' sizes are taken from the kernel's source."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "compressed_sparse_attention_07_gb300",
                      "csrc", "kv_tiles.cu")
STAGES, WARPS = 2, 4  # of operands; of keys or of values


def _constants():
    text = open(SOURCE).read()
    return {n: int(re.search(r"\b%s = (\d+)" % n, text).group(1)) for n in ("kRing", "kLongRing", "kStages")}


class Wrong(Exception):
    pass


def _check(ok, what):
    if not ok:
        raise Wrong(what)


class Barrier:
    def __init__(self, arrivals):
        self.arrivals, self.here, self.phase = arrivals, 0, 0

    def arrive(self):
        self.here += 1
        if self.here == self.arrivals:
            self.here, self.phase = 0, self.phase + 1


def _wait(bar, use):
    """Until the phase with the parity of `use` is over; it has to be that very one."""
    while (bar.phase & 1) == (use & 1):
        yield
    _check(bar.phase > use, "a wait passed on an earlier phase")
    _check(bar.phase <= use + 1, "a phase ran past a warp that waits for it")


class Model:
    """n tiles through the kernel; ring: places of undecoded tiles (0: pages are copied as they are); turns: one tile of
    rows, whose places take the key tiles in turn."""

    def __init__(self, seed, n, ring, turns):
        self.rnd, self.n, self.ring, self.turns = random.Random(seed), n, ring, turns
        self.full = {v: [Barrier(1 if v and not ring else WARPS) for _ in range(STAGES)] for v in (0, 1)}
        self.free = {v: [Barrier(1) for _ in range(STAGES)] for v in (0, 1)}
        self.s_ready, self.p_ready, self.o_full = [Barrier(1), Barrier(1)], [Barrier(2), Barrier(2)], [Barrier(1), Barrier(1)]
        self.raw_full, self.raw_free = [Barrier(1) for _ in range(ring)], [Barrier(WARPS) for _ in range(ring)]
        self.raw, self.stage = [None] * ring, {}
        self.scores, self.weights, self.summed = [None, None], [(-1, 0), (-1, 0)], [-1, -1]
        self.flying, self.issued = [], []

    # -- the warps, each a generator that yields where another may run
    def fetch(self, v):
        for it in range(self.n):
            op = 2 * it + v
            slot = op % self.ring
            if op >= self.ring:
                yield from _wait(self.raw_free[slot], op // self.ring - 1)
            self.raw[slot] = None

            def land(slot=slot, op=op):
                self.raw[slot] = op
                self.raw_full[slot].arrive()
            self.flying.append(land)
            yield

    def decode(self, v, w):
        for it in range(self.n):
            op = 2 * it + v
            slot, s = op % self.ring, it % STAGES
            yield from _wait(self.raw_full[slot], op // self.ring)
            _check(self.raw[slot] == op, "an undecoded tile read before it had landed")
            yield
            _check(self.raw[slot] == op, "an undecoded tile overwritten while it was read")
            self.raw_free[slot].arrive()
            yield from self.written(v, w, it)
            self.full[v][s].arrive()

    def copy(self, v, w):
        for it in range(self.n):
            yield from self.written(v, w, it, -1)

            def land(it=it):
                self.stage[v, w, it % STAGES] = it
                self.full[v][it % STAGES].arrive()
            self.flying.append(land)
            yield

    def written(self, v, w, it, value=None):
        if it >= STAGES:
            yield from _wait(self.free[v][it % STAGES], it // STAGES - 1)
        self.stage[v, w, it % STAGES] = it if value is None else value
        yield

    def operand(self, v, it):
        for w in range(WARPS if self.ring or not v else 1):
            _check(self.stage.get((v, w, it % STAGES)) == it, "a product read %s of another tile" % ("values" if v else "keys"))

    def product_scores(self, j, it, u, over):
        def run():
            self.operand(0, it)
            _check(u == 0 or self.summed[j] == u - 1, "scores over weights that were not used up")
            self.scores[j] = u
        self.issued += [run, self.s_ready[j].arrive] + ([self.free[0][it % STAGES].arrive] if over else [])

    def product_outputs(self, j, it, u, done):
        def run():
            self.operand(1, it)
            _check(self.weights[j] == (u, 2), "weights read before they were written")
            self.summed[j] = u
        self.issued += [run] + ([done.arrive] if done else [])

    def issue(self):
        n, full, free = self.n, self.full, self.free
        if self.turns:
            for it in range(n):
                s = it % 2
                yield from _wait(full[0][s], it // STAGES)
                if it >= 2:
                    yield from _wait(full[1][s], it // STAGES - 1)
                    yield from _wait(self.p_ready[s], it // 2 - 1)
                    self.product_outputs(s, it - 2, it // 2 - 1, free[1][s])
                self.product_scores(s, it, it // 2, True)
                yield
            for it in range(max(0, n - 2), n):
                yield from _wait(full[1][it % 2], it // STAGES)
                yield from _wait(self.p_ready[it % 2], it // 2)
                self.product_outputs(it % 2, it, it // 2, self.o_full[it % 2])
        else:
            for it in range(n):
                s, p = it % STAGES, (it - 1) % STAGES
                yield from _wait(full[0][s], it // STAGES)
                for j in (0, 1):
                    if it > 0:
                        if j == 0:
                            yield from _wait(full[1][p], (it - 1) // STAGES)
                        yield from _wait(self.p_ready[j], it - 1)
                        self.product_outputs(j, it - 1, it - 1, free[1][p] if j else None)
                    self.product_scores(j, it, it, j == 1)
                    yield
            if n:
                yield from _wait(full[1][(n - 1) % STAGES], (n - 1) // STAGES)
                for j in (0, 1):
                    yield from _wait(self.p_ready[j], n - 1)
                    self.product_outputs(j, n - 1, n - 1, self.o_full[j])

    def soft(self, j):
        tiles = range(j, self.n, 2) if self.turns else range(self.n)
        for u, _ in enumerate(tiles):
            yield from _wait(self.s_ready[j], u)
            _check(self.scores[j] == u, "scores of another tile")
            yield
            last, some = self.weights[j]
            self.weights[j] = (u, some + 1 if last == u else 1)
            self.p_ready[j].arrive()
            yield
        for k in (0, 1) if self.turns else (j,):
            count = len(range(k, self.n, 2)) if self.turns else self.n
            if count:
                yield from _wait(self.o_full[k], 0)
                _check(self.summed[k] == count - 1, "outputs read before the last product")

    def run(self):
        if self.ring:
            warps = [self.decode(v, w) for v in (0, 1) for w in range(WARPS)] + [self.fetch(0), self.fetch(1)]
        else:
            warps = [self.copy(0, w) for w in range(WARPS)] + [self.copy(1, 0)]
        warps += [self.soft(j) for j in (0, 1) for _ in range(2)] + [self.issue()]
        weight = [self.rnd.choice((1, 1, 3, 10)) for _ in warps]
        for _ in range(200000):
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
                    return
        raise Wrong("a standstill")


def _failures(ring, turns, seeds):
    wrong = []
    for seed in range(seeds):
        n = random.Random(seed).choice((0, 1, 2, 3, 4, 5, 9, 20))
        try:
            Model(seed, n, ring, turns).run()
        except Wrong as e:
            wrong.append("%d tiles, seed %d: %s" % (n, seed, e))
    return wrong


@pytest.mark.parametrize("ring,turns", [("kRing", False), ("kLongRing", True), (None, False), (None, True)])
def test_no_schedule_goes_wrong(ring, turns):
    c = _constants()
    assert c["kStages"] == STAGES
    assert not _failures(c[ring] if ring else 0, turns, 150)


@pytest.mark.parametrize("ring", [3, 5])
@pytest.mark.parametrize("turns", [False, True])
def test_a_ring_of_odd_size_is_found_wrong(ring, turns):
    """Keys and values alternate: with an odd number of places a warp sees every second phase of each, and the parity of
    one that is over is that of the one it waits for."""
    assert _failures(ring, turns, 60)
