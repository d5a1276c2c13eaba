"""The ring that holds rows in shared memory (csrc/rowring.cuh), on the host: the
order of its loads, waits and arrivals as the kernels' warps go through them, with
the arithmetic they use (csrc/ringorder.h), under schedules that hold any one warp
or copy back as long as something else can run.

A wait on an mbarrier tells only even phases from odd ones.  So a warp must see each
load of a slot while it is the slot's latest: if the next one can land before a warp
has looked, that warp's wait is for a phase that has gone by, and it waits for ever."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HELD = 4         # rows between a sum and its output
WARPS = 2        # sum warps, and output warps


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    so = tmp_path_factory.mktemp("ring") / "ring_order.so"
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC",
                    "-I" + os.path.join(ROOT, "greedy_spec_decode_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "host", "ring_order.cpp"), "-o", str(so)],
                   check=True, capture_output=True, text=True)
    return ctypes.CDLL(str(so))


class Barrier:
    """An mbarrier: `count` arrivals (or a landed copy) end a phase."""

    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self, n=1):
        assert n <= self.pending, "more arrivals than the phase has"
        self.pending -= n
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def passes(self, parity):
        return (self.phase & 1) != parity


class Model:
    """One CTA that takes rows of stages[i] stages each through a ring of `slots`."""

    def __init__(self, ring, slots, stages):
        self.ring, self.slots, self.stages = ring, slots, stages
        self.full = [Barrier(1) for _ in range(slots)]
        self.empty = [Barrier(ring.ring_arrivals(WARPS)) for _ in range(slots)]
        self.stored = [Barrier(WARPS) for _ in range(HELD)]
        self.told = [0] * len(stages)
        self.joined = [0] * len(stages)
        self.landing = []        # slots with a copy in flight
        self.done = 0

    def loads(self, it):
        return self.ring.ring_loads(self.stages[it], self.slots, 1)

    def see(self, at, load):
        """A wait for load number `load` of all: yields until the barrier lets it by."""
        slot, parity = at >> 1, at & 1
        assert slot == load % self.slots and parity == load // self.slots % 2
        while not self.full[slot].passes(parity):
            yield False
        assert self.full[slot].phase == load // self.slots + 1, "another load was taken for it"
        yield True

    def copies(self):
        at = filled = 0
        for it in range(len(self.stages)):
            for _ in range(self.loads(it)):
                slot = at >> 1
                if filled < self.slots:
                    filled += 1
                else:
                    while not self.empty[slot].passes((at & 1) ^ 1):
                        yield False
                assert slot not in self.landing
                self.landing.append(slot)
                at = self.ring.ring_step(at, self.slots)
                yield True

    def lands(self, slot):
        while True:
            while slot not in self.landing:
                yield False
            self.landing.remove(slot)
            self.full[slot].arrive()
            yield True

    def sums(self, warp):
        at, base = 0, 0
        for it, stages in enumerate(self.stages):
            r = at
            for j in range(self.loads(it)):
                if j == stages:
                    yield from self.join(it, warp)
                yield from self.see(r, base + j)
                n = self.ring.ring_sum_arrivals(j, stages, self.slots)
                if n:
                    self.empty[r >> 1].arrive(n)
                r = self.ring.ring_step(r, self.slots)
            if self.loads(it) == stages:
                yield from self.join(it, warp)
            at = self.ring.ring_later(at, self.loads(it), self.slots)
            base += self.loads(it)

    def join(self, it, warp):
        self.joined[it] += 1
        while self.joined[it] < WARPS:
            yield False
        if warp == it % WARPS:
            if it >= HELD:
                while not self.stored[it % HELD].passes((it // HELD - 1) & 1):
                    yield False
                assert self.stored[it % HELD].phase == it // HELD
            self.told[it] = 1
        yield True

    def outputs(self, warp):
        at, base = 0, 0
        for it, stages in enumerate(self.stages):
            while not self.told[it]:
                yield False
            kept = max(0, stages - self.slots)
            r = self.ring.ring_later(at, kept, self.slots)
            for i in range(stages):
                yield from self.see(r, base + kept + i)
                self.empty[r >> 1].arrive()
                r = self.ring.ring_step(r, self.slots)
            self.stored[it % HELD].arrive()
            yield True
            at = self.ring.ring_later(at, self.loads(it), self.slots)
            base += self.loads(it)

    def run(self, rng, last):
        """Runs everything, agent `last` only when nothing else can."""
        work = [self.copies()] + [self.sums(w) for w in range(WARPS)] + \
            [self.outputs(w) for w in range(WARPS)]
        agents = work + [self.lands(s) for s in range(self.slots)]
        open_ = set(range(len(work)))
        while open_:
            order = list(range(len(agents)))
            rng.shuffle(order)
            order.sort(key=lambda a: a == last)
            for a in order:
                if a < len(work) and a not in open_:
                    continue
                try:
                    if next(agents[a]):
                        break
                except StopIteration:
                    open_.discard(a)
                    break
            else:
                raise AssertionError(f"nothing can run: {sorted(open_)} wait for ever")


AGENTS = 1 + 2 * WARPS


@pytest.mark.parametrize("slots,stages", [
    (3, [1, 3, 2, 0, 3, 1, 2, 3]),               # rows that the ring holds
    (3, [4, 4, 4, 4, 4, 4]), (3, [5, 1, 6, 3, 4, 9, 2]), (4, [9, 9, 9, 9, 9, 9]),
    (3, [3, 7, 3, 7, 4, 20, 1]), (5, [6, 11, 10, 9, 5, 6, 16])], ids=str)
def test_every_warp_sees_every_load(ring, slots, stages):
    for last in [None] + list(range(AGENTS + slots)):
        for seed in range(12):
            Model(ring, slots, stages).run(random.Random(seed), last)
