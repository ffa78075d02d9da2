"""Host-side model of k_tree_attn's barrier protocol (w12_attn.cu; no GPU).

Producer warps fill a ring of K and V tiles, one warp issues the scores, one the outputs, softmax
warps stand between the two.  A wait for the k-th completion of an mbarrier is a parity wait: it is exact
only if, whenever it looks, the barrier has completed k or k + 1 phases.  One behind, it passes
on an older phase; one ahead, it misses the phase and stalls.

The simulation gives every copy, product and step of a warp a random time, with heavy tails (a warp may be
held for longer than all others' work of a unit), and checks every look of every wait.  The planted case
waits for the last unit's end behind a unit's scores instead of in front of the last hand-over: that
unit may then have ended too, and the phase is missed.
"""
import heapq
import random

import pytest

PLANS = {64: (10, 3, True), 128: (5, 3, True), 256: (5, 4, False)}  # ring slots, score buffers, two tiles of rows


class Stale(Exception):
    pass


class Sim:
    def __init__(self, rng):
        self.rng, self.now, self.seq, self.heap = rng, 0.0, 0, []
        self.count, self.arrived, self.done, self.waiters, self.running = {}, {}, {}, {}, 0

    def time(self, lo, hi):
        t = self.rng.uniform(lo, hi)
        return t * 10 if self.rng.random() < 0.05 else t

    def look(self):
        """Until a warp looks at a barrier."""
        return self.rng.uniform(5, 30) if self.rng.random() < 0.02 else self.rng.uniform(0.01, 0.1)

    def at(self, t, fn):
        self.seq += 1
        heapq.heappush(self.heap, (t, self.seq, fn))

    def arrive(self, bar):
        n = self.arrived.get(bar, 0) + 1
        if n < self.count.get(bar[0], 1):
            self.arrived[bar] = n
            return
        self.arrived[bar] = 0
        self.done[bar] = self.done.get(bar, 0) + 1
        for actor in self.waiters.pop(bar, []):
            self.at(self.now + self.look(), lambda a=actor: self.step(*a))

    def start(self, gen):
        self.running += 1
        self.at(self.time(0, 1), lambda: self.step(gen, None))

    def step(self, gen, waiting):
        """Advances an actor; it yields a time to sleep or a (barrier, phase) to wait for."""
        if waiting:
            bar, k = waiting
            done = self.done.get(bar, 0)
            if done not in (k, k + 1):
                raise Stale(f"{bar}: waits for phase {k}, {done} completed")
            if done == k:
                self.waiters.setdefault(bar, []).append((gen, waiting))
                return
        try:
            what = next(gen)
        except StopIteration:
            self.running -= 1
            return
        wait = None if isinstance(what, float) else what
        self.at(self.now + (self.look() if wait else what), lambda: self.step(gen, wait))

    def run(self):
        while self.heap:
            self.now, _, fn = heapq.heappop(self.heap)
            fn()
        assert self.running == 0, "stalled"


def ring_tile(item, cnt, two):
    if two:
        return item >> 1, bool(item & 1)
    if item == 2 * cnt - 1:
        return cnt - 1, True
    if item < 2:
        return item, False
    is_v = not item & 1
    return ((item - 2) >> 1 if is_v else (item + 1) >> 1), is_v


def ring_item(tile, is_v, cnt, two):
    if two:
        return 2 * tile + is_v
    if is_v:
        return 2 * cnt - 1 if tile == cnt - 1 else 2 * tile + 2
    return tile if tile < 2 else 2 * tile - 1


PRODUCERS, QUARTERS = 2, 2


def kernel(rng, plan, units, late=False):
    slots, buffers, _ = plan
    sim = Sim(rng)
    sim.count = dict(full=PRODUCERS, q_full=PRODUCERS, reset=PRODUCERS, meta=PRODUCERS, pair=2, p_full=2 * QUARTERS,
                     unit_end=2 * QUARTERS)
    after = lambda t, bar: sim.at(sim.now + t, lambda: sim.arrive(bar))
    bufs = lambda two: (1, 2) if two else tuple(range(buffers))

    def producer():
        entry = 0
        for u, (cnt, two) in enumerate(units):
            for item in range(2 * cnt):
                slot, turn = entry % slots, entry // slots
                entry += 1
                if turn:
                    yield ("empty", slot), turn - 1
                yield sim.time(0.1, 0.5)
                after(sim.time(0.5, 3), ("full", slot))
                if item == 0:
                    if u:
                        yield ("q_free",), u - 1
                    after(sim.time(0.5, 3), ("q_full",))
                    sim.arrive(("reset",))
                    yield ("reset",), u
                    yield sim.time(0.1, 0.5)
                    sim.arrive(("meta", u & 1))

    class Products:
        """Products of one warp: they end in any order, a commit arrives when all before it have."""

        def __init__(self):
            self.end = 0.0

        def issue(self):
            self.end = max(self.end, sim.now + sim.time(0.3, 1))

        def commit(self, bar):
            sim.at(max(self.end, sim.now), lambda: sim.arrive(bar))

    def scores():
        entry, used, outputs, had_two, mma = 0, set(), [0] * buffers, False, Products()
        for u, (cnt, two) in enumerate(units):
            yield ("q_full",), u
            ended = u == 0
            if had_two and not two and not ended:
                yield ("unit_end",), u - 1
                ended = True
            had_two = two
            steps = 2 * cnt if two else cnt
            for x in range(steps):
                row_tile, tile = (x & 1, x >> 1) if two else (0, x)
                b = bufs(two)[x % len(bufs(two))]
                if b in used:
                    yield ("o_done", b), outputs[b]
                    outputs[b] += 1
                used.add(b)
                if not row_tile:
                    e = entry + ring_item(tile, False, cnt, two)
                    yield ("full", e % slots), e // slots
                yield sim.time(0.05, 0.3)
                mma.issue()
                if not late and x == steps - 1 and not ended:
                    yield ("unit_end",), u - 1
                mma.commit(("s_full", b))
                if not two or row_tile:
                    mma.commit(("empty", e % slots))
            if late and not ended:
                yield ("unit_end",), u - 1
            mma.commit(("q_free",))
            entry += 2 * cnt

    def outputs():
        entry, seen, mma = 0, [0] * buffers, Products()
        for u, (cnt, two) in enumerate(units):
            if u:
                yield ("unit_end",), u - 1
            for x in range(2 * cnt if two else cnt):
                row_tile, tile = (x & 1, x >> 1) if two else (0, x)
                b = bufs(two)[x % len(bufs(two))]
                yield ("p_full", b), seen[b]
                seen[b] += 1
                if not row_tile:
                    e = entry + ring_item(tile, True, cnt, two)
                    yield ("full", e % slots), e // slots
                yield sim.time(0.05, 0.3)
                mma.issue()
                mma.commit(("o_done", b))
                if not two or row_tile:
                    mma.commit(("empty", e % slots))
            entry += 2 * cnt

    def softmax(quarter):
        seen, ends, told = [0] * buffers, [0] * buffers, 0

        def done(b):
            ends[b] += 1
            return ("o_done", b), ends[b] - 1

        for u, (cnt, two) in enumerate(units):
            yield ("meta", u & 1), u >> 1
            order, last = bufs(two), 0
            steps = 2 * cnt if two else cnt
            for x in range(steps):
                b = order[x % len(order)]
                last = b if two else last
                yield ("s_full", b), seen[b]
                seen[b] += 1
                sim.arrive(("pair", quarter))
                yield ("pair", quarter), told
                told += 1
                early = sim.rng.random() < 0.3
                first = (x >> 1 if two else x) == 0
                if early and not first:
                    yield done(last)
                yield sim.time(0.5, 1.5)
                if not early and not first:
                    yield done(last)
                sim.arrive(("p_full", b))
                last = b
            yield done(order[0] if two else last)
            if two:
                yield done(order[1])
            for _ in range(2 if two else 1):
                sim.arrive(("pair", quarter))
                yield ("pair", quarter), told
                told += 1
            yield sim.time(0.2, 1)
            sim.arrive(("unit_end",))

    for _ in range(PRODUCERS):
        sim.start(producer())
    sim.start(scores())
    sim.start(outputs())
    for q in range(QUARTERS):
        for _ in range(2):
            sim.start(softmax(q))
    sim.run()


def share(rng, plan):
    most = rng.choice([1, 2, 3, 7, 20])
    return [(rng.randint(1, most), plan[2] and rng.random() < 0.4) for _ in range(rng.randint(1, 12))]


@pytest.mark.parametrize("d", sorted(PLANS))
def test_ring_order_and_its_inverse(d):
    for two in (False, True):
        for cnt in range(1, 12):
            order = [ring_tile(i, cnt, two) for i in range(2 * cnt)]
            assert sorted(order) == sorted((t, v) for t in range(cnt) for v in (False, True))
            assert [ring_item(t, v, cnt, two) for t, v in order] == list(range(2 * cnt))


@pytest.mark.parametrize("d", sorted(PLANS))
def test_every_phase_is_waited_for(d):
    for seed in range(400):
        rng = random.Random(seed)
        kernel(rng, PLANS[d], share(rng, PLANS[d]))


@pytest.mark.parametrize("d", sorted(PLANS))
def test_a_late_wait_for_a_unit_s_end_misses_it(d):
    stale = 0
    for seed in range(400):
        rng = random.Random(seed)
        try:
            kernel(rng, PLANS[d], share(rng, PLANS[d]), late=True)
        except Stale as e:
            assert "unit_end" in str(e)
            stale += 1
    assert stale
