"""The barriers of the block-sparse backward, restated: agents that wait for and arrive on barriers
with phases, as the kernels' warps do, under random times of loads and products.  No agent may
touch a buffer that does not hold what it expects.  The numbers of the barriers are the kernel
source's own."""
import heapq
import os
import random
import re

import pytest

SOURCE = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                           "persistent_sm_attn_b200", "csrc", "sparse_bwd.cuh")).read()


class Barrier:
    """An mbarrier: a phase ends with `count` arrivals; wait(parity) passes once the phase of that
    parity is over, that is while the current phase has the other one."""

    def __init__(self, count=1):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def over(self, parity):
        return (self.phase & 1) != parity


class Machine:
    """Agents are generators that yield a delay, or a (barrier, parity) to wait for."""

    def __init__(self, agents):
        self.now, self.order, self.heap, self.blocked = 0.0, 0, [], []
        for a in agents:
            self.at(0.0, a)

    def at(self, t, what):
        self.order += 1
        heapq.heappush(self.heap, (t, self.order, what))

    def later(self, dt, fn):
        self.at(self.now + dt, fn)

    def step(self, agent):
        while True:
            try:
                y = next(agent)
            except StopIteration:
                return
            if isinstance(y, tuple):
                if not y[0].over(y[1]):
                    self.blocked.append((y, agent))
                    return
            else:
                self.at(self.now + y, agent)
                return

    def run(self):
        while self.heap:
            self.now, _, what = heapq.heappop(self.heap)
            if callable(what):
                what()
            else:
                self.step(what)
            again = True
            while again:
                again = False
                for item in list(self.blocked):
                    (bar, parity), agent = item
                    if bar.over(parity):
                        self.blocked.remove(item)
                        self.step(agent)
                        again = True
        assert not self.blocked, "the agents wait for one another"


def dq_pass(seed, barriers, units=40, kK=6, kV=4):
    """dQ of one tile.  Returns the units whose S or dP was taken before it was there."""
    rng = random.Random(seed)
    bad = []
    K_FULL, K_EMPTY = [Barrier() for _ in range(kK)], [Barrier() for _ in range(kK)]
    V_FULL, V_EMPTY = [Barrier() for _ in range(kV)], [Barrier() for _ in range(kV)]
    S_FULL, DP_FULL = [Barrier() for _ in range(barriers)], [Barrier() for _ in range(barriers)]
    DS_READY = [Barrier() for _ in range(3)]
    s_in, dp_in = [None] * 3, [None] * 3
    ph = lambda j, n: (j // n) & 1
    slow = lambda: rng.expovariate(1.0) * rng.choice([1, 1, 1, 100])  # a load, now and then a late one

    def producer():
        for j in range(units):
            if j >= kK:
                yield K_EMPTY[j % kK], ph(j - kK, kK)
            m.later(slow(), K_FULL[j % kK].arrive)
            if j >= kV:
                yield V_EMPTY[j % kV], ph(j - kV, kV)
            m.later(slow(), V_FULL[j % kV].arrive)
            yield 0.01

    def scores(first):
        for j in range(first, units, 2):
            yield K_FULL[j % kK], ph(j, kK)
            if j >= 3:
                yield K_EMPTY[(j - 3) % kK], ph(j - 3, kK)
            yield 0.3
            s_in[j % 3] = j
            S_FULL[j % barriers].arrive()
            yield V_FULL[j % kV], ph(j, kV)
            yield 0.3
            dp_in[j % 3] = j
            DP_FULL[j % barriers].arrive()
            V_EMPTY[j % kV].arrive()

    def softmax(first):
        for j in range(first, units, 2):
            yield S_FULL[j % barriers], ph(j, barriers)
            if s_in[j % 3] != j:
                bad.append(j)
            yield 0.4
            yield DP_FULL[j % barriers], ph(j, barriers)
            if dp_in[j % 3] != j:
                bad.append(j)
            yield 0.4
            DS_READY[j % 3].arrive()

    def gradient():
        for j in range(units):
            yield DS_READY[j % 3], ph(j, 3)
            yield 0.3
            K_EMPTY[j % kK].arrive()

    m = Machine([producer(), scores(0), scores(1), softmax(0), softmax(1), gradient()])
    try:
        m.run()
    except AssertionError:
        bad.append(None)
    return bad


@pytest.mark.parametrize("stages", [(6, 4), (8, 8)])
def test_dq_takes_no_scores_before_they_are_there(stages):
    n, = set(re.findall(r"auto (?:S_FULL|DP_FULL) = \[&\]\(int j\) \{ return bar2[^;]*\(j % (\d)\)", SOURCE))
    for seed in range(300):
        assert dq_pass(seed, int(n), kK=stages[0], kV=stages[1]) == [], seed
    # one barrier a buffer is not enough: two warpgroups' phases take turns on it
    assert any(dq_pass(seed, 3, kK=stages[0], kV=stages[1]) for seed in range(300))


def dkdv_pass(seed, dv_waits_for_dp, tiles=40, stages=2):
    """dK and dV of one item at D = 128.  Returns the tiles whose dO was read by dV or dP when the
    stage held another, or replaced while dP still read it."""
    rng = random.Random(seed)
    bad = []
    FULL = [[Barrier() for _ in range(stages)] for _ in range(2)]   # Q, dO
    EMPTY = [[Barrier() for _ in range(stages)] for _ in range(2)]
    S_FULL, DP_FULL, SDP_READ, P_READY, P_FREE, DS_READY, DS_FREE = (
        [Barrier(), Barrier()] for _ in range(7))
    held, reading = [None] * stages, [None] * stages   # tile whose dO a stage holds; that dP reads
    ph = lambda j, n: (j // n) & 1
    slow = lambda: rng.expovariate(1.0) * rng.choice([1, 1, 1, 30])

    def loader(x):
        for j in range(tiles):
            s = j % stages
            if j >= stages:
                yield EMPTY[x][s], ph(j - stages, stages)
            if x:
                if reading[s] is not None:
                    bad.append(reading[s])
                held[s] = None
            yield slow()
            if x:
                held[s] = j
            FULL[x][s].arrive()

    def scores():
        for j in range(tiles):
            s = j % stages
            yield FULL[0][s], ph(j, stages)
            if j >= 2:
                yield SDP_READ[j % 2], ph(j - 2, 2)
            yield 0.3
            S_FULL[j % 2].arrive()
            yield rng.choice([0, 0, 3])  # another warp's thread is late now and then
            yield FULL[1][s], ph(j, stages)
            if held[s] != j:
                bad.append(j)
            reading[s] = j
            yield 0.3
            if held[s] != j:
                bad.append(j)
            reading[s] = None
            DP_FULL[j % 2].arrive()

    def softmax():
        for j in range(tiles):
            yield S_FULL[j % 2], ph(j, 2)
            yield 0.4
            if j:
                yield P_FREE[(j - 1) % 2], ph(j - 1, 2)
            P_READY[j % 2].arrive()
            yield DP_FULL[j % 2], ph(j, 2)
            if j:
                yield DS_FREE[(j - 1) % 2], ph(j - 1, 2)
            yield 0.4
            SDP_READ[j % 2].arrive()
            DS_READY[j % 2].arrive()

    def gradients():
        for j in range(tiles):
            s = j % stages
            if dv_waits_for_dp:
                yield DP_FULL[j % 2], ph(j, 2)
            yield P_READY[j % 2], ph(j, 2)
            if held[s] != j:
                bad.append(j)
            yield 0.3
            P_FREE[j % 2].arrive()
            EMPTY[1][s].arrive()
            yield DS_READY[j % 2], ph(j, 2)
            yield 0.3
            EMPTY[0][s].arrive()
            DS_FREE[j % 2].arrive()

    m = Machine([loader(0), loader(1), scores(), softmax(), gradients()])
    try:
        m.run()
    except AssertionError:
        bad.append(None)
    return bad


def test_dv_reads_and_frees_a_stage_of_dO_after_dP():
    waits = "wait(DP_FULL(j), ph2(j)) && wait(P_READY(j), ph2(j))" in SOURCE
    for seed in range(300):
        assert dkdv_pass(seed, waits) == [], seed
    assert any(dkdv_pass(seed, False) for seed in range(300))
