"""CPU: the ring of linear_int8 as a state machine. Barriers have phases, and a wait names one by its
parity; a producer fills places, copies land in any order, two groups of four warps take the stages in
turn and release them, and MMAs complete in order behind them. Steps are taken in a random order,
with copies and warps held back at random. No warp may read a place before its own stage's copy has landed
there, and no copy may be announced in a phase that has one already or over a place that is still read."""
import os
import random
import re

import pytest

from conftest import ROOT

WARPS = 4  # of each of the two groups


def depths():
    """The rings' depths by rows of a tile: int8_stages() of the host's plan."""
    with open(os.path.join(ROOT, "dense_gemm_gb300", "csrc", "ops.cu")) as f:
        body = re.search(r"constexpr int int8_stages\(int T\) \{ return ([^;]*); \}", f.read()).group(1)
    found = [int(n) for n in re.findall(r"\? (\d+)|: (\d+)$", body) for n in n if n]
    assert len(found) == 3, body
    return sorted(set(found))


class Fault(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phases = self.bytes = 0

    def settle(self):
        if self.left == 0 and self.bytes == 0:
            self.left = self.count
            self.phases += 1

    def arrive(self):
        if self.left == 0:
            raise Fault("an arrival too many in one phase")
        self.left -= 1
        self.settle()

    def expect(self):
        if self.left == 0:
            raise Fault("two copies announced in one phase")
        self.bytes += 1
        self.arrive()

    def land(self):
        self.bytes -= 1
        self.settle()

    def passes(self, parity):
        """try_wait.parity: the phase of that parity, or the one before the current, is over."""
        return self.phases % 2 != parity


def run(stages, steps, second_wait, seed):
    rng = random.Random(seed)
    full = [Barrier(1) for _ in range(stages)]
    empty = [Barrier(WARPS) for _ in range(stages)]
    ready, used = [Barrier(WARPS) for _ in range(2)], [Barrier(1) for _ in range(2)]
    holds = [None] * stages       # the stage whose bytes lie in a place
    flying, mmas = [], []         # copies on their way; MMAs that have not completed
    readers = [0] * stages        # warps that have a place's current stage still to read

    def announce(st):
        place = st % stages
        if readers[place]:
            raise Fault("a copy over a place that is still read")
        full[place].expect()
        flying.append(st)
        readers[place] = WARPS

    def producer():
        for st in range(min(stages, steps)):
            announce(st)
            yield None
        place = phase = 0
        for st in range(stages, steps):
            yield lambda p=place, q=phase: empty[p].passes(q)
            announce(st)
            place += 1
            if place == stages:
                place, phase = 0, phase ^ 1

    def warp(group):
        place, phase, turn = group, 0, 0
        for st in range(group, steps, 2):
            if second_wait and stages % 2 and st >= stages:
                yield lambda p=place, q=phase ^ 1: empty[p].passes(q)
            yield lambda p=place, q=phase: full[p].passes(q)
            yield lambda q=turn ^ 1: used[group].passes(q)
            if holds[place] != st:
                raise Fault(f"stage {st} is read where {holds[place]} lies")
            yield None
            if holds[place] != st:
                raise Fault(f"stage {st} was overwritten while it was read")
            readers[place] -= 1
            empty[place].arrive()
            yield None
            ready[group].arrive()
            place += 2
            if place >= stages:
                place, phase = place - stages, phase ^ 1
            turn ^= 1

    def issuer():
        c = turn = 0
        for _ in range(steps):
            yield lambda c=c, q=turn: ready[c].passes(q)
            mmas.append(c)
            turn ^= c
            c ^= 1

    class Actor:
        def __init__(self, steps_):
            self.steps, self.wait, self.done, self.weight = steps_, None, False, rng.choice((0.05, 1.0, 1.0))

        def can(self):
            return not self.done and (self.wait is None or self.wait())

        def step(self):
            try:
                self.wait = next(self.steps)
            except StopIteration:
                self.done = True

    actors = [Actor(producer()), Actor(issuer())] + [Actor(warp(g)) for g in (0, 1) for _ in range(WARPS)]
    slow = rng.choice((0.02, 0.2, 1.0))  # copies against warps
    late = {}                            # how long a copy is held back against the others
    while not all(a.done for a in actors) or flying or mmas:
        choices = [(a.weight, a.step) for a in actors if a.can()]
        for st in flying:
            def land(st=st):
                flying.remove(st)
                holds[st % stages] = st
                full[st % stages].land()
            choices.append((slow * late.setdefault(st, rng.choice((0.01, 1.0))), land))
        if mmas:
            choices.append((0.5, lambda: used[mmas.pop(0)].arrive()))
        if not choices:
            raise Fault("all wait")
        weights, moves = zip(*choices)
        rng.choices(moves, weights)[0]()


@pytest.mark.parametrize("stages", sorted(set(depths()) | {2, 3, 4, 5, 6}))
def test_every_order_reads_its_own_stage(stages):
    for seed in range(120):
        run(stages, random.Random(seed).choice((1, 2, stages, 3 * stages + 1, 40)), True, seed)


def test_rings_that_are_used():
    assert depths() == [3, 4, 6]


@pytest.mark.parametrize("stages", [3])
def test_odd_rings_need_the_release(stages):
    """Without the wait for the other group's release some orders read a place too early."""
    faults = set()
    for seed in range(400):
        try:
            run(stages, 40, False, seed)
        except Fault as e:
            faults.add(str(e).split(" ")[0])
    assert faults


@pytest.mark.parametrize("stages", [2, 4, 6])
def test_even_rings_do_not(stages):
    for seed in range(120):
        run(stages, 40, False, seed)
