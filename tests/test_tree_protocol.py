"""A model of the tree attention kernel's pipeline on the CPU: loader, MMA
issuers and row warps as coroutines with random speeds and random delays of copies
and MMAs, over the kernel's barriers (phases seen by their parity alone) and
ring.  What it must never see: a barrier with more arrivals than it counts, a slot
or tile read that holds something else than the reader wants, a stop.  The
model follows csrc/tree.cu by hand; ring sizes are read from it."""
from __future__ import annotations

import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_grouped_expert_gb300", "csrc",
                   "tree.cu")


def ring_slots(D):
    m = re.search(r"NS = D == 256 \? (\d+) : D == 128 \? (\d+) : (\d+);", open(SRC).read())
    return int(m.group({256: 1, 128: 2, 64: 3}[D]))


class Bar:
    def __init__(self, count, name):
        self.count, self.pending, self.phase, self.name = count, count, 0, name

    def arrive(self):
        assert self.pending > 0, f"{self.name}: too many arrivals"
        self.pending -= 1
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def done(self, parity):  # what a wait on a parity sees
        return (self.phase & 1) != (parity & 1)


class Model:
    def __init__(self, seed, units, slots, parts, warps, two, active, edge, slow, ahead_of_output=2):
        self.r = random.Random(seed)
        self.units, self.slots, self.parts, self.warps, self.two = units, slots, parts, warps, two
        self.active, self.edge, self.slow, self.bound = active, edge, slow, ahead_of_output
        bars = lambda n, c, name: [Bar(c, f"{name}{i}") for i in range(n)]  # noqa: E731
        self.full, self.empty = bars(slots, 1, "full"), bars(slots, 1, "empty")
        self.p_ready, self.pv_done, self.pair = bars(2, warps, "p_ready"), bars(2, 1, "pv_done"), bars(4, 2, "pair")
        self.s_full, self.s_free, self.q_full, self.q_free = (Bar(1, "s_full"), Bar(warps, "s_free"), Bar(1, "q_full"),
                                                              Bar(1, "q_free"))
        self.o_free, self.rows_bar = Bar(warps, "o_free"), Bar(warps, "rows")
        self.tag, self.landing, self.s_mma = [None] * slots, [], []
        self.o_mma = [] if two else self.s_mma
        self.S = self.O = self.Q = None
        self.P = [None, None]
        self.grows = [self.r.random() < 0.15 for _ in range(sum(units) + 1)]

    def k_pos(self, j):
        return self.parts * (0 if j == 0 else 2 * j - 1)

    def v_pos(self, j, n):
        return self.parts * (2 * n - 1 if j == n - 1 else 2 * j + 2)

    def wait(self, bar, phase):
        while not bar.done(phase):
            yield

    def slot(self, pos, want):
        s = pos % self.slots
        yield from self.wait(self.full[s], pos // self.slots)
        assert self.tag[s] == want, f"slot holds {self.tag[s]}, wanted {want}"

    def loader(self):
        ld = 0
        for u, n in enumerate(self.units):
            if u:
                yield from self.wait(self.q_free, u - 1)
            self.Q = None
            self.land(lambda u=u: (setattr(self, "Q", u), self.q_full.arrive()))
            order = [("K", 0)] + [x for j in range(n) for x in ([("K", j + 1)] if j + 1 < n else []) + [("V", j)]]
            for kind, j in order:
                for part in range(self.parts):
                    s = ld % self.slots
                    yield from self.wait(self.empty[s], ld // self.slots + 1)
                    assert self.full[s].phase == ld // self.slots, "a load into a slot whose last one is under way"
                    self.tag[s] = "loading"
                    self.land(lambda s=s, t=(kind, u, j, part): (self.tag.__setitem__(s, t), self.full[s].arrive()))
                    ld += 1

    def land(self, f):
        self.landing.append([self.r.randint(1, self.slow if self.r.random() < 0.1 else 8), f])

    def scores(self, u, j, ld, t):
        if t >= 1:
            yield from self.wait(self.s_free, t - 1)
        if self.bound and j == 0 and t >= 2:
            yield from self.wait(self.pv_done[t & 1], (t - 2) >> 1)
        for part in range(self.parts):
            pos, want = ld + self.k_pos(j) + part, ("K", u, j, part)
            yield from self.slot(pos, want)

            def run(s=pos % self.slots, want=want, last=part == self.parts - 1):
                assert self.tag[s] == want and self.Q == u
                self.empty[s].arrive()
                if last:
                    self.S = t
                    self.s_full.arrive()
            self.s_mma.append(run)
            yield

    def values(self, u, j, n, ld, t):
        yield from self.wait(self.p_ready[t & 1], t >> 1)
        if j == 0 and u:
            yield from self.wait(self.o_free, u - 1)
        for part in range(self.parts):
            pos, want = ld + self.v_pos(j, n) + part, ("V", u, j, part)
            yield from self.slot(pos, want)

            def run(s=pos % self.slots, want=want, last=part == self.parts - 1):
                assert self.tag[s] == want and self.P[t & 1] == t
                self.empty[s].arrive()
                if last:
                    self.O = t
                    self.pv_done[t & 1].arrive()
            self.o_mma.append(run)
            yield

    def issuer(self, does_s, does_o):
        ld = t = 0
        for u, n in enumerate(self.units):
            if does_s:
                yield from self.wait(self.q_full, u)
                yield from self.scores(u, 0, ld, t)
            for j in range(n):
                if does_s:
                    if j + 1 < n:
                        yield from self.scores(u, j + 1, ld, t + 1)
                    if j + 1 == max(1, n - 1):
                        self.s_mma.append(self.q_free.arrive)
                if does_o:
                    yield from self.values(u, j, n, ld, t)
                t += 1
            ld += 2 * self.parts * n

    def row_warp(self, w):
        ld = t = pairs = syncs = 0
        for u, n in enumerate(self.units + [0]):
            if u:  # the result of the unit before
                yield from self.wait(self.pv_done[(t - 1) & 1], (t - 1) >> 1)
                assert self.O == t - 1, "a result taken out too early"
                if self.warps == 8:
                    self.pair[w % 4].arrive()
                    pairs += 1
                    yield from self.wait(self.pair[w % 4], pairs - 1)
                self.o_free.arrive()
            for j in range(n):
                if j == max(0, n - self.edge[u]):
                    for _ in range(2):
                        self.rows_bar.arrive()
                        syncs += 1
                        yield from self.wait(self.rows_bar, syncs - 1)
                yield from self.wait(self.s_full, t)
                assert self.S == t
                if self.bound and t >= 2:
                    yield from self.wait(self.pv_done[t & 1], (t - 2) >> 1)
                if j >= n - self.edge[u]:
                    if self.bound and t >= 1:
                        yield from self.wait(self.pv_done[(t - 1) & 1], (t - 1) >> 1)
                    for part in range(self.parts):
                        yield from self.slot(ld + self.v_pos(j, n) + part, ("V", u, j, part))
                if self.active[u][w]:
                    for _ in range(self.r.randint(0, 4)):
                        yield
                    assert self.S == t, "scores overwritten before they were read"
                    self.s_free.arrive()
                    if self.warps == 8:
                        self.pair[w % 4].arrive()
                        pairs += 1
                        yield from self.wait(self.pair[w % 4], pairs - 1)
                    if j and self.grows[t]:
                        yield from self.wait(self.pv_done[(t - 1) & 1], (t - 1) >> 1)
                        assert self.O == t - 1
                    for _ in range(self.r.randint(2, 20)):
                        yield
                    if not self.bound and t >= 2:
                        yield from self.wait(self.pv_done[t & 1], (t - 2) >> 1)
                    self.P[t & 1] = t
                else:
                    self.s_free.arrive()
                yield
                self.p_ready[t & 1].arrive()
                t += 1
            ld += 2 * self.parts * n

    def run(self):
        roles = [self.loader()] + ([self.issuer(True, False), self.issuer(False, True)] if self.two
                                   else [self.issuer(True, True)]) + [self.row_warp(w) for w in range(self.warps)]
        speed = [self.r.choice([0.15, 0.5, 0.9]) for _ in roles]
        alive, cool, steps = set(range(len(roles))), [0, 0], 0
        queues = [self.s_mma, self.o_mma] if self.two else [self.s_mma]
        while alive or self.landing or any(queues):
            for i in sorted(alive):
                if self.r.random() < speed[i]:
                    try:
                        next(roles[i])
                    except StopIteration:
                        alive.discard(i)
            for x in self.landing[:]:
                x[0] -= 1
                if x[0] <= 0:
                    self.landing.remove(x)
                    x[1]()
            for i, q in enumerate(queues):
                cool[i] -= 1
                if q and cool[i] <= 0:
                    q.pop(0)()
                    cool[i] = self.r.randint(1, 8)
            steps += 1
            assert steps < 4000 + 3000 * sum(self.units), "the pipeline stopped"


def model(seed, D, **kw):
    r = random.Random(seed)
    units = [r.choice([1, 1, 2, 3, 4, 5, 9, 17]) for _ in range(r.randint(1, 5))]
    warps = 8 if D == 256 else 4
    active = [[w % 4 < k for w in range(warps)] for k in (r.randint(1, 4) for _ in units)]
    edge = [r.randint(0, min(n, 3)) for n in units] + [0]
    return Model(seed, units, ring_slots(D), 2 if D == 256 else 1, warps, D == 256, active, edge,
                 r.choice([10, 60, 300]), **kw)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_pipeline_never_stops_or_reads_a_wrong_slot(D):
    for seed in range(150):
        model(seed, D).run()


def test_the_model_sees_a_missing_wait():
    # without the bound on how far rows may be ahead of the output
    with pytest.raises(AssertionError):
        for seed in range(150):
            model(seed, 256, ahead_of_output=0).run()
