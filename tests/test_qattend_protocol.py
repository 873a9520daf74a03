"""Models of the pipelines of attention over the 8-bit cache on the CPU: loaders, MMA
issuers and row warps as coroutines with random speeds and random delays of copies
and MMAs, over the kernels' barriers (phases seen by their parity alone) and rings.  What
they must never see: a barrier with more arrivals than it counts, a slot, tile or exchanged
value that is another than the reader wants, a stop.  (The wait for o_free alone is implied by p_ready, for
which every row warp arrives after it.)  The models follow csrc/qattend.cu (rows in
the lanes) and csrc/qdecode.cu (positions in the lanes) by hand; ring sizes are read from there."""
from __future__ import annotations

import os
import random
import re

import pytest

from tests.test_tree_protocol import Bar

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_grouped_expert_gb300", "csrc")
WARPS = 8


def rings(name, D, parts):
    """Slots of K, of V and of the scales."""
    text, pick = open(os.path.join(SRC, name)).read(), {256: 1, 128: 2, 64: 3}[D]
    k = int(re.search(r"NSK = D == 256 \? (\d+) : D == 128 \? (\d+) : (\d+)", text).group(pick))
    v = re.search(r"NSV = D == 256 \? (5 - PARTS|\d+) : NSK", text).group(1)
    s = (re.search(r"SCALES = D == 256 \? (\d+) : D == 128 \? (\d+) : (\d+)", text) if name == "qattend.cu" else None)
    if s:
        scales = int(s.group(pick))
    else:
        at64, others = map(int, re.search(r"SCALES = D == 64 \? (\d+) : (\d+)", text).groups())
        scales = at64 if D == 64 else others
    return k, (5 - parts if v == "5 - PARTS" else int(v)) if D == 256 else k, scales


class Model:
    """What both kernels have: the rings, copies that land and MMAs that end when they like."""

    def __init__(self, seed, units, edge, slots, slow, leave_out=""):
        self.r, self.units, self.edge, self.slow, self.out = random.Random(seed), units, edge, slow, leave_out
        self.nsk, self.nsv, self.nsc = slots
        self.full = {"K": self.bars(self.nsk, 1, "k_full"), "V": self.bars(self.nsv, 1, "v_full")}
        self.empty = {"K": self.bars(self.nsk, 1, "k_empty"), "V": self.bars(self.nsv, 1, "v_empty")}
        self.sc_full = self.bars(self.nsc, 1, "sc_full")
        self.tag = {"K": [None] * self.nsk, "V": [None] * self.nsv}
        self.scales = [None] * self.nsc
        self.landing, self.s_mma, self.o_mma = [], [], []
        self.q_full, self.o_free, self.O = None, Bar(WARPS, "o_free"), None
        self.tiles = sum(units)

    @staticmethod
    def bars(n, count, name):
        return [Bar(count, f"{name}{i}") for i in range(n)]

    def wait(self, bar, phase, name=""):
        if name and name == self.out:  # a wait that a test leaves out
            return
        while not bar.done(phase):
            yield

    def pause(self, most):
        for _ in range(self.r.randint(0, most)):
            yield

    def land(self, f):
        self.landing.append([self.r.randint(1, self.slow if self.r.random() < 0.1 else 8), f])

    def loader(self, kind):
        n, t = len(self.full[kind]), 0
        for u, tiles in enumerate(self.units):
            if kind == "V":
                yield from self.queries(u)
            for _ in range(tiles):
                s = t % n
                yield from self.wait(self.empty[kind][s], t // n + 1)
                assert self.full[kind][s].phase == t // n, "a load into a slot whose last one is under way"
                self.tag[kind][s] = "loading"
                self.land(lambda s=s, t=t: (self.tag[kind].__setitem__(s, t), self.full[kind][s].arrive()))
                if kind == "K":
                    i = t % self.nsc
                    self.scales[i] = "loading"
                    self.land(lambda i=i, t=t: (self.scales.__setitem__(i, t), self.sc_full[i].arrive()))
                t += 1
                yield

    def queries(self, u):
        return iter(())

    def run(self):
        roles = [self.loader("K"), self.loader("V"), self.issue_s(), self.issue_o()] + [self.row_warp(w) for w in range(WARPS)]
        speed = [self.r.choice([0.15, 0.5, 0.9]) for _ in roles]
        alive, cool, steps = set(range(len(roles))), [0, 0], 0
        while alive or self.landing or self.s_mma or self.o_mma:
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
            for i, q in enumerate((self.s_mma, self.o_mma)):
                cool[i] -= 1
                if q and cool[i] <= 0:
                    q.pop(0)()
                    cool[i] = self.r.randint(1, 8)
            steps += 1
            assert steps < 4000 + 3000 * self.tiles, "the pipeline stopped"


class Rows(Model):
    """qattend.cu: one S and one P tile, queries by TMA."""

    def __init__(self, seed, units, edge, slots, slow, active, leave_out=""):
        super().__init__(seed, units, edge, slots, slow, leave_out)
        self.active = active
        self.q_full, self.q_free = Bar(1, "q_full"), Bar(1, "q_free")
        self.s_full, self.s_free, self.p_ready, self.pv_done = (Bar(1, "s_full"), Bar(WARPS, "s_free"), Bar(WARPS, "p_ready"),
                                                                Bar(1, "pv_done"))
        self.pair = self.bars(4, 2, "pair")
        self.S = self.Q = None
        self.P, self.row = [None] * WARPS, [[None] * WARPS for _ in range(2)]

    def queries(self, u):
        if u:
            yield from self.wait(self.q_free, u - 1, "q_free")
        self.Q = None
        self.land(lambda: (setattr(self, "Q", u), self.q_full.arrive()))

    def issue_s(self):
        t = 0

        def scores(t, u):
            if t:
                yield from self.wait(self.s_free, t - 1, "s_free")
            s = t % self.nsk
            yield from self.wait(self.full["K"][s], t // self.nsk)

            def run():
                assert self.tag["K"][s] == t and self.Q == u, "an S over other keys or queries"
                self.S = t
                self.empty["K"][s].arrive()
                self.s_full.arrive()
            self.s_mma.append(run)
            yield

        for u, n in enumerate(self.units):
            yield from self.wait(self.q_full, u)
            yield from scores(t, u)
            for j in range(n):
                if j + 1 < n:
                    yield from scores(t + 1, u)
                if j + 1 == max(1, n - 1):
                    self.s_mma.append(self.q_free.arrive)
                t += 1

    def issue_o(self):
        t = 0
        for u, n in enumerate(self.units):
            for j in range(n):
                yield from self.wait(self.p_ready, t)
                if j == 0 and u:
                    yield from self.wait(self.o_free, u - 1, "o_free")
                s = t % self.nsv
                yield from self.wait(self.full["V"][s], t // self.nsv)

                def run(s=s, t=t):
                    assert self.tag["V"][s] == t and self.P == [t] * WARPS, "an O over other values or weights"
                    self.O = t
                    self.empty["V"][s].arrive()
                    self.pv_done.arrive()
                self.o_mma.append(run)
                yield
                t += 1

    def row_warp(self, w):
        t = pairs = 0

        def exchange(value):
            nonlocal pairs
            turn = pairs & 1
            self.row[turn][w] = value
            yield
            self.pair[w % 4].arrive()
            pairs += 1
            yield from self.wait(self.pair[w % 4], pairs - 1)
            yield from self.pause(4)
            assert self.row[turn][w ^ 4] == value, "another exchange's value"

        for u, n in enumerate(self.units + [0]):
            if u:  # the result of the unit before
                yield from self.wait(self.pv_done, t - 1, "result")
                assert self.O == t - 1, "a result taken out too early"
                yield from exchange(("maximum", u))
                yield from exchange(("sum", u))
                yield from self.pause(10)
                assert self.O == t - 1, "a result overwritten"
                self.o_free.arrive()
            for j in range(n):
                yield from self.wait(self.s_full, t)
                yield from self.wait(self.sc_full[t % self.nsc], t // self.nsc)
                assert self.S == t
                if j >= n - self.edge[u]:
                    s = t % self.nsv
                    yield from self.wait(self.full["V"][s], t // self.nsv)
                    assert self.tag["V"][s] == t, "values that are not this tile's cleared"
                if self.active[u][w]:
                    yield from self.pause(4)
                    assert self.S == t, "scores overwritten before they were read"
                    self.s_free.arrive()
                    yield from self.pause(12)
                    assert self.scales[t % self.nsc] == t, "scales overwritten before they were read"
                    yield from exchange(("score", t))
                    yield from self.pause(20)
                    if t:
                        yield from self.wait(self.pv_done, t - 1, "active")
                        assert self.O == t - 1, "O changed before its product"
                    self.P[w] = t
                else:
                    self.s_free.arrive()
                    if t:
                        yield from self.wait(self.pv_done, t - 1, "inactive")
                    self.P[w] = t
                yield
                self.p_ready.arrive()
                t += 1


class Positions(Model):
    """qdecode.cu: two S and two P tiles, queries cut by the row warps."""

    def __init__(self, seed, units, edge, slots, slow, leave_out=""):
        super().__init__(seed, units, edge, slots, slow, leave_out)
        self.q_full = Bar(WARPS, "q_full")
        two = lambda count, name: self.bars(2, count, name)  # noqa: E731
        self.s_full, self.s_free, self.p_ready, self.pv_done, self.met = (two(1, "s_full"), two(WARPS, "s_free"),
                                                                          two(WARPS, "p_ready"), two(1, "pv_done"), two(4, "meet"))
        self.Q, self.S, self.P = [None] * WARPS, [None, None], [[None] * WARPS for _ in range(2)]
        self.factor = [[None] * WARPS for _ in range(4)]
        self.flag = [[None] * WARPS for _ in range(2)]
        self.most, self.sums = [None] * WARPS, [None] * WARPS
        self.grows = [[self.r.random() < 0.3 for _ in range(self.tiles + 1)] for _ in range(2)]

    def issue_s(self):
        t = 0

        def scores(t, u):
            if t >= 2:
                yield from self.wait(self.s_free[t & 1], (t - 2) >> 1, "s_free")
            s = t % self.nsk
            yield from self.wait(self.full["K"][s], t // self.nsk)

            def run():
                assert self.tag["K"][s] == t and self.Q == [u] * WARPS, "an S over other keys or queries"
                self.S[t & 1] = t
                self.empty["K"][s].arrive()
                self.s_full[t & 1].arrive()
            self.s_mma.append(run)
            yield

        for u, n in enumerate(self.units):
            yield from self.wait(self.q_full, u)
            yield from scores(t, u)
            for j in range(n):
                if j + 1 < n:
                    yield from scores(t + 1, u)
                t += 1

    def issue_o(self):
        t = 0
        for u, n in enumerate(self.units):
            for j in range(n):
                yield from self.wait(self.p_ready[t & 1], t >> 1)
                if j == 0 and u:
                    yield from self.wait(self.o_free, u - 1, "o_free")
                s = t % self.nsv
                yield from self.wait(self.full["V"][s], t // self.nsv)

                def run(s=s, t=t):
                    assert self.tag["V"][s] == t and self.P[t & 1] == [t] * WARPS, "an O over other values or weights"
                    self.O = t
                    self.empty["V"][s].arrive()
                    self.pv_done[t & 1].arrive()
                self.o_mma.append(run)
                yield
                t += 1

    def row_warp(self, w):
        half, t, meets = w // 4, 0, 0
        mine = slice(4 * half, 4 * half + 4)

        def meet():
            nonlocal meets
            yield
            self.met[half].arrive()
            meets += 1
            yield from self.wait(self.met[half], meets - 1)

        def cut(u):
            yield from self.pause(8)
            self.Q[w] = u
            self.factor[u & 3][w] = u
            self.q_full.arrive()

        yield from cut(0)
        for u, n in enumerate(self.units):
            for j in range(n):
                yield from self.wait(self.s_full[t & 1], t >> 1)
                yield from self.wait(self.pv_done[t & 1], (t >> 1) - 1 if t >= 2 else 1, "p_tile")
                yield from self.wait(self.sc_full[t % self.nsc], t // self.nsc)
                assert self.S[t & 1] == t
                if j >= n - self.edge[u]:
                    s = t % self.nsv
                    yield from self.wait(self.full["V"][s], t // self.nsv)
                    assert self.tag["V"][s] == t, "values that are not this tile's cleared"
                assert self.scales[t % self.nsc] == t, "scales overwritten before they were read"
                yield from self.pause(4)
                assert self.S[t & 1] == t and self.factor[u & 3] == [u] * WARPS and self.scales[t % self.nsc] == t
                self.s_free[t & 1].arrive()
                if j == n - 1 and u + 1 < len(self.units):
                    yield from cut(u + 1)
                yield from self.pause(4)
                self.flag[t & 1][w] = t
                yield from meet()
                yield from self.pause(4)
                assert self.flag[t & 1][mine] == [t] * 4, "another tile's flags"
                up = self.grows[half][t] or j == 0
                if up:
                    self.most[w] = t
                    yield from meet()
                    yield from self.pause(4)
                    assert self.most[mine] == [t] * 4, "another tile's maxima"
                yield from self.pause(10)
                self.P[t & 1][w] = t
                if up and j:
                    yield from self.wait(self.pv_done[(t - 1) & 1], (t - 1) >> 1, "rescale")
                    assert self.O == t - 1, "O changed before its product"
                    yield
                    assert self.O == t - 1
                self.p_ready[t & 1].arrive()
                t += 1
            self.sums[w] = u
            yield from meet()
            yield from self.pause(4)
            assert self.sums[mine] == [u] * 4, "another unit's sums"
            yield from self.wait(self.pv_done[(t - 1) & 1], (t - 1) >> 1, "result")
            assert self.O == t - 1, "a result taken out too early"
            yield from self.pause(10)
            assert self.O == t - 1, "a result overwritten"
            self.o_free.arrive()


def rows(seed, D, parts, leave_out=""):
    r = random.Random(seed)
    units = [r.choice([1, 1, 2, 3, 4, 5, 9, 17]) for _ in range(r.randint(1, 5))]
    edge = [r.randint(0, min(n, 3)) for n in units]
    active = [[w % 4 < k for w in range(WARPS)] for k in (r.randint(1, 4) for _ in units)]
    return Rows(seed, units, edge, rings("qattend.cu", D, parts), r.choice([10, 60, 300]), active, leave_out)


def positions(seed, D, leave_out=""):
    r = random.Random(seed)
    units = [r.choice([1, 1, 2, 3, 4, 5, 9, 17]) for _ in range(r.randint(1, 6))]
    edge = [r.randint(0, min(n, 3)) for n in units]
    return Positions(seed, units, edge, rings("qdecode.cu", D, 3), r.choice([10, 60, 300]), leave_out)


@pytest.mark.parametrize("D,parts", [(64, 2), (128, 3), (256, 2), (256, 3)])
def test_rows_in_the_lanes_never_stop_or_read_what_is_not_theirs(D, parts):
    for seed in range(150):
        rows(seed, D, parts).run()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_positions_in_the_lanes_never_stop_or_read_what_is_not_theirs(D):
    for seed in range(150):
        positions(seed, D).run()


@pytest.mark.parametrize("wait", ["q_free", "s_free", "result", "active", "inactive"])
def test_the_model_of_rows_sees_a_missing_wait(wait):
    with pytest.raises(AssertionError):
        for seed in range(150):
            rows(seed, 256, 2, wait).run()


@pytest.mark.parametrize("wait", ["s_free", "result", "p_tile", "rescale"])
def test_the_model_of_positions_sees_a_missing_wait(wait):
    with pytest.raises(AssertionError):
        for seed in range(150):
            positions(seed, 256, wait).run()
