"""The barrier protocol of the attention mass above 128 query rows, as a
discrete-event model (no GPU): a producer, two warps that issue the row tiles
in turn, the -lse warp and two groups of row warps, with the waits, phases and
barrier counts of mla_mass_rows_kernel.  Waits are parity waits, as the
hardware's: a wait for phase k also passes while phase k - 2 was the last one
to complete, so a barrier may only be waited on where that cannot be.

The model shows why score tiles need six barriers (three let a group pass the
wait for tile j while tile j - 3 was still on its way), and that six suffice.
"""
import heapq
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_mla_decode_09_gb300", "csrc",
                      "mla_mass.cu")
SLOTS, FULL = 3, 6  # ring slots, barriers of its entries
SCORES = 3          # score buffers


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count

    def passed(self, k):  # the parity wait for phase k
        return (self.phase & 1) != (k & 1)


class Model:
    def __init__(self, bars, tiles, units, land):
        self.t, self.events, self.order = 0, [], 0
        self.kv_full = [Bar(1) for _ in range(FULL)]
        self.s_full = [Bar(2) for _ in range(bars)]
        self.s_empty = [Bar(1) for _ in range(SCORES)]
        self.q_full, self.q_bar = Bar(2), [Bar(1), Bar(1)]
        self.bars, self.tiles, self.units, self.land = bars, tiles, units, land
        self.holds = [None] * SCORES     # the tile whose scores a buffer holds in full
        self.slots = [None] * SLOTS      # the entry that a slot holds
        self.faults = []
        self.busy = 0                    # until when the tensor pipe has work

    def at(self, dt, fn):
        self.order += 1
        heapq.heappush(self.events, (self.t + dt, self.order, fn))

    def run(self):
        procs = [self.produce(), self.issue(0), self.issue(1), self.lse(), self.rows(0), self.rows(1)]
        waiting = {}
        ready = list(enumerate(procs))
        left = len(procs)
        while True:
            while ready:
                n, g = ready.pop(0)
                try:
                    what = next(g)
                except StopIteration:
                    left -= 1
                    continue
                if isinstance(what, tuple):
                    waiting[n] = (g, what)
                else:
                    self.at(what, lambda n=n, g=g: ready.append((n, g)))
            for n in list(waiting):
                g, (bar, k) = waiting[n]
                if bar.passed(k):
                    del waiting[n]
                    ready.append((n, g))
            if ready:
                continue
            if not self.events:
                if left:
                    self.faults.append("stalled")
                return self.faults
            self.t, _, fn = heapq.heappop(self.events)
            fn()

    def s_wait(self, j):
        return self.s_full[j % self.bars], j // self.bars

    def produce(self):
        i = j = 0
        held = []
        for u in range(self.units):
            for e in range(2):
                if len(held) >= SLOTS:
                    kind, k = held[-SLOTS]
                    yield (self.q_full, k) if kind == "keys" else self.s_wait(k)
                held.append(("keys", u))
                self.kv_full[i % FULL].arrive()
                if e == 1:
                    self.at(self.land(), lambda u=u: self.q_bar[u & 1].arrive())
                i += 1
            for _ in range(self.tiles):
                if len(held) >= SLOTS:
                    kind, k = held[-SLOTS]
                    yield (self.q_full, k) if kind == "keys" else self.s_wait(k)
                held.append(("tile", j))
                self.slots[i % SLOTS] = j

                def landed(i=i):
                    self.kv_full[i % FULL].arrive()

                self.at(self.land(), landed)
                i += 1
                j += 1
            yield 1

    def issue(self, w):
        i = j = 0
        for u in range(self.units):
            i += 2
            yield self.q_full, u
            for _ in range(self.tiles):
                if j & 1 == w:
                    yield self.kv_full[i % FULL], i // FULL
                    yield self.s_empty[j % SCORES], j // SCORES + 1  # free: parity of the phase before
                    if self.slots[i % SLOTS] != j:
                        self.faults.append(f"tile {j} issued from another entry")
                    self.holds[j % SCORES] = None
                    self.busy = max(self.busy, self.t) + 1224

                    def done(j=j):
                        self.holds[j % SCORES] = j
                        self.s_full[j % self.bars].arrive()

                    self.at(self.busy - self.t, done)
                    yield 230
                i += 1
                j += 1

    def lse(self):
        j = 0
        for _ in range(self.units * self.tiles):
            yield self.s_empty[j % SCORES], j // SCORES + 1
            self.s_full[j % self.bars].arrive()
            j += 1
            yield 20

    def rows(self, g):
        j = 0
        for u in range(self.units):
            for back in (1, 2):
                if j >= back:
                    yield self.s_wait(j - back)
            yield self.q_bar[u & 1], u >> 1
            yield 500
            self.q_full.arrive()
            for _ in range(self.tiles):
                if j & 1 == g:
                    yield self.s_wait(j)
                    if self.holds[j % SCORES] != j:
                        self.faults.append(f"group {g} read tile {j} where buffer held {self.holds[j % SCORES]}")
                    yield 150
                    self.s_empty[j % SCORES].arrive()
                    yield 500
                j += 1


def faults(bars, seed):
    rng = random.Random(seed)
    slow = rng.choice([0.0, 0.02, 0.2, 0.5])
    late = rng.choice([1500, 4000, 12000])
    m = Model(bars, rng.choice([3, 4, 5, 6, 9, 16, 64]), rng.choice([1, 2, 3, 7]),
              lambda: rng.randint(700, 1100) + (rng.randint(0, late) if rng.random() < slow else 0))
    return m.run()


def test_three_barriers_for_three_buffers_are_too_few():
    assert any(faults(3, seed) for seed in range(300))


@pytest.mark.parametrize("part", range(4))
def test_the_kernels_barriers_never_let_a_tile_pass(part):
    with open(SOURCE) as f:
        bars = int(re.search(r"constexpr int kScoreFull = (\d+);", f.read()).group(1))
    for seed in range(1000 * part, 1000 * part + 1000):
        assert faults(bars, seed) == [], (bars, seed)
