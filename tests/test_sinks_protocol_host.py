"""Race check, on the CPU, of the barrier protocol of the window-plus-sinks
prefill kernels, with the model of test_barrier_protocols_host.py.

They wait for P_{j-1} V_{j-1} only where they need O (to rescale it, and for the
output): S_j's commit covers P_{j-2} V_{j-2} and all before. There is one P-ready
barrier per buffer of P. k_prefill_stream also walks several row tiles
without a pause: Q is loaded again when the row tile's last S is done (q_empty),
and the output of a row tile is taken out of TMEM after the first softmax of the
next one, whose first P V waits for that (o_free). With one row tile the model
is k_prefill_tc's and k_prefill_pair's.
"""
import random

import pytest

from test_barrier_protocols_host import KERNELS, Bar, Model

KERNELS.update({
    "sinks": dict(n_cta=1, smem_p=False, per_buffer=True, pv_before_arrive=False),
    "sinks_pair": dict(n_cta=2, smem_p=False, per_buffer=True, pv_before_arrive=False),
    "sinks_one_p_ready": dict(n_cta=1, smem_p=False, per_buffer=False, pv_before_arrive=False),
})


class Stream(Model):
    """Row tiles of `row_tiles` key tiles each, one after the other."""

    def __init__(self, kernel, row_tiles, KS, VS, NSTAGE, rng, skip=()):
        super().__init__(kernel, sum(row_tiles), KS, VS, NSTAGE, rng, skip)
        self.rows = row_tiles
        self.q_empty = [Bar("q_empty/cta%d" % c, 1) for c in range(self.C)]
        self.o_free = Bar("o_free", self.C)
        self.out = [[] for _ in range(self.C)]
        self.first = {}   # key tile -> its row tile's number, for first tiles
        self.last = {}
        t = 0
        for n, k in enumerate(row_tiles):
            self.first[t], self.last[t + k - 1] = n, n
            t += k

    def q_inflight(self, c):
        return any(res == ("Q", c) for res, _ in self.tma_inflight)

    def producer(self, c):
        item = 0

        def load(n_stages):
            nonlocal item
            for _ in range(n_stages):
                s = item % self.NS
                if item >= self.NS:
                    while not self.check_wait(self.empty[c][s], item // self.NS - 1, "empty"):
                        yield
                if self.reads(("stage", c, s)):
                    self.hazard("copy into stage %d of CTA %d while an MMA reads it" % (s, c))
                if c == 0 and self.C > 1:
                    self.full[s].arrive()  # arm
                self.tma_inflight.append((("stage", c, s), self.full[s]))
                item += 1
                yield

        def load_q():
            if self.reads(("Q", c)):
                self.hazard("copy into Q of CTA %d while an MMA reads it" % c)
            if c == 0 and self.C > 1:
                self.q_full.arrive()
            self.tma_inflight.append((("Q", c), self.q_full))

        load_q()
        for j in range(self.n):
            yield from load(self.KS)
            if j > 0:
                yield from load(self.VS)
            n = self.first.get(j, 0)
            if n > 0:
                while not self.check_wait(self.q_empty[c], n - 1, "q_empty"):
                    yield
                load_q()
        yield from load(self.VS)

    def issuer(self):
        C = range(self.C)
        item = 0

        def pv(t):
            nonlocal item
            n = self.first.get(t, 0)
            if n > 0:
                while not self.check_wait(self.o_free, n - 1, "o_free"):
                    yield
                for c in C:
                    if n - 1 not in self.out[c]:
                        self.hazard("PV_%d issued before CTA %d took output %d" % (t, c, n - 1))
            bar, k = (self.p_ready[t & 1], t >> 1) if self.per_buffer else (self.p_ready[0], t)
            while not self.check_wait(bar, k, "p_ready"):
                yield
            for c in C:
                if t not in self.p_written[c]:
                    self.hazard("PV_%d issued before CTA %d wrote P_%d" % (t, c, t))
            for _ in range(self.VS):
                s = item % self.NS
                while not self.check_wait(self.full[s], item // self.NS, "full"):
                    yield
                self.tc_queue.append(("mma", ("PV", t), {("stage", c, s) for c in C} | {self.p_res(c, t) for c in C},
                                      {("O", c) for c in C}))
                self.tc_queue.append(("commit", [self.empty[c][s] for c in C], None))
                item += 1
                yield
            self.tc_queue.append(("commit", [self.o_done[c][t & 1] for c in C], ("PV", t)))

        for j in range(self.n):
            if j in self.first:
                while not self.check_wait(self.q_full, self.first[j], "q_full"):
                    yield
                for c in C:
                    if self.q_inflight(c):
                        self.hazard("S_%d issued with Q of CTA %d on its way" % (j, c))
            for c in C:
                if j >= 2 and (j - 2) not in self.s_read[c]:
                    self.hazard("S_%d issued over S_%d before CTA %d read it" % (j, j - 2, c))
            for _ in range(self.KS):
                s = item % self.NS
                while not self.check_wait(self.full[s], item // self.NS, "full"):
                    yield
                self.tc_queue.append(("mma", ("S", j), {("stage", c, s) for c in C} | {("Q", c) for c in C},
                                      {("S", c, j & 1) for c in C}))
                self.tc_queue.append(("commit", [self.empty[c][s] for c in C], None))
                item += 1
                yield
            self.tc_queue.append(("commit", [self.s_full[c][j & 1] for c in C], ("S", j)))
            if j in self.last:
                self.tc_queue.append(("commit", self.q_empty, None))
            yield
            if j >= 1:
                yield from pv(j - 1)
        yield from pv(self.n - 1)

    def softmax(self, c):
        def pv_done(t, role):
            while not self.check_wait(self.o_done[c][t & 1], t >> 1, role):
                yield

        def put_out(t):
            if t not in self.pv_done or self.writes(("O", c)):
                self.hazard("CTA %d took the output after tile %d with a PV product in flight" % (c, t))
            self.out[c].append(self.last[t])
            self.o_free.arrive()

        for j in range(self.n):
            while not self.check_wait(self.s_full[c][j & 1], j >> 1, "s_full"):
                yield
            if j not in self.s_done or self.writes(("S", c, j & 1)):
                self.hazard("CTA %d read S_%d with its MMA not complete" % (c, j))
            self.s_read[c].add(j)
            yield
            if j not in self.first and self.rng.random() < 0.4:  # rescale O
                yield from pv_done(j - 1, "rescale")
                if self.writes(("O", c)) or self.reads(("O", c)):
                    self.hazard("CTA %d rescaled O with a PV product in flight (tile %d)" % (c, j))
                yield
            res = self.p_res(c, j)
            if self.reads(res) or self.writes(res):
                self.hazard("CTA %d wrote P_%d over a buffer an MMA still uses" % (c, j))
            self.p_written[c].add(j)
            (self.p_ready[j & 1] if self.per_buffer else self.p_ready[0]).arrive()
            yield
            if j > 0 and j in self.first:
                yield from pv_done(j - 1, "pv_done")
                put_out(j - 1)
                yield
        yield from pv_done(self.n - 1, "pv_done")
        put_out(self.n - 1)


# row tiles, K and V stages of a key tile, ring stages: the stream kernel (1, 1, 4), the
# pair at head_dim 512 (2, 1, 3), the single CTA at 256 (2, 2, 5) and 512 (4, 2, 3), and rings
# as short as the order allows
SHAPES = {
    "sinks": [((1,), 2, 2, 5), ((2,), 2, 2, 5), ((7,), 2, 2, 5), ((6,), 4, 2, 3), ((1, 1, 1), 1, 1, 3),
              ((3, 1, 4), 1, 1, 4)],
    "sinks_pair": [((1,), 2, 1, 3), ((5,), 2, 1, 3), ((4, 1, 1, 3), 1, 1, 4), ((2, 2, 2), 1, 1, 4), ((1, 1, 1, 1), 1, 1, 4),
                   ((3, 5), 1, 1, 3)],
}


def violations(kernel, shape, seeds, skip=()):
    for seed in range(seeds):
        m = Stream(kernel, *shape, rng=random.Random(seed), skip=skip)
        m.run()
        if m.violations:
            return m.violations
    return []


@pytest.mark.parametrize("kernel,shape", [(k, s) for k in SHAPES for s in SHAPES[k]])
def test_protocol_has_no_race(kernel, shape):
    assert not violations(kernel, shape, 150)


@pytest.mark.parametrize("wait", ["empty", "full", "q_full", "q_empty", "o_free", "s_full", "p_ready", "pv_done", "rescale"])
def test_each_wait_is_needed(wait):
    assert violations("sinks_pair", ((3, 2, 4), 1, 1, 4), 300, skip=(wait,))


def test_one_p_ready_barrier_would_not_do():
    assert violations("sinks_one_p_ready", ((8,), 1, 1, 4), 300)
