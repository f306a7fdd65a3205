"""A model check of the RMSNorm gradient's ring of bulk copies (CPU).

train_rms_grad_ring_kernel's first thread fetches a row per stage, every thread waits for the stage,
works on it, and behind the block's barrier the first thread fetches the stage's next row.  A
wait has a limit; one that gives up sets the abort flag, after which every wait gives up at once.
This module restates that (in ends.cu's order) with copies that land at random times or, in part
of the runs, not before the block has ended, and waits that may give up, and checks that a stage
is never fetched into while copies into it are outstanding and that no barrier phase receives
more arrivals than it expects.  Keep it in step with ends.cu."""
import random

import pytest

from test_attention_protocol import Sim

THREADS = 3


class Ring:
    def __init__(self, rows, stages, late, check_abort, seed):
        self.rnd = random.Random(seed)
        self.rows, self.stages, self.late, self.check_abort = rows, stages, late, check_abort
        self.sim = Sim()
        self.out = [0] * stages          # copies under way into the stage
        self.abort = False
        self.bars = [self.sim.bar(s) for s in range(stages)]
        self.fetched = 0

    def fetch(self, row, st):
        assert self.out[st] == 0, "a stage is fetched into while a copy into it is under way"
        self.bars[st].expect_tx(2)
        self.fetched += 1
        for _ in range(2):               # x and grad_y
            self.out[st] += 1

            def land(st=st):
                self.out[st] -= 1
                self.bars[st].complete_tx(1)
            if not (self.late and row == self.late and self.rnd.random() < 0.7):
                self.sim.events.append(land)

    def land_some(self, all_of_them=False):
        while self.sim.events and (all_of_them or self.rnd.random() < 0.6):
            self.sim.events.pop(self.rnd.randrange(len(self.sim.events)))()

    def wait(self, st, parity):
        """One thread's wait: False if it gives up."""
        if self.abort:
            return False
        for _ in range(50):
            if self.bars[st].done(parity):
                return True
            self.land_some()
        self.abort = True
        return False

    def run(self):
        arrived = []
        for i in range(self.stages):
            if i < self.rows:
                self.fetch(i, i)
        st = phase = 0
        for row in range(self.rows):
            arrived.append(all([self.wait(st, phase) for _ in range(THREADS)]))
            # the block's barrier, then the first thread
            if row + self.stages < self.rows and not (self.check_abort and self.abort):
                self.fetch(row + self.stages, st)
            st += 1
            if st == self.stages:
                st, phase = 0, phase ^ 1
        return arrived


@pytest.mark.parametrize("stages", [2, 3, 8])
@pytest.mark.parametrize("rows", [1, 2, 7, 20])
def test_every_row_arrives(stages, rows):
    for seed in range(30):
        r = Ring(rows, stages, 0, True, seed)
        assert r.run() == [True] * rows
        assert r.fetched == rows and not r.abort


@pytest.mark.parametrize("stages", [2, 3, 8])
def test_nothing_is_fetched_after_a_wait_gave_up(stages):
    gave_up = 0
    for seed in range(60):
        r = Ring(20, stages, 1 + seed % 15, True, seed)
        arrived = r.run()
        if r.abort:
            gave_up += 1
            first = arrived.index(False)
            assert not any(arrived[first:]), "a row counts as arrived after a wait gave up"
            assert r.fetched <= first + stages
    assert gave_up > 20


def test_planted_fetch_after_a_wait_gave_up_is_caught():
    caught = 0
    for seed in range(60):
        try:
            Ring(20, 2, 1 + seed % 15, False, seed).run()
        except AssertionError:
            caught += 1
    assert caught > 20
