"""A model of how the gated recurrence's CTAs exchange their maps (csrc/glr.cu: send, receive,
exchange_end) under waits that give up at any time.

Each CTA sends the map of a round to every CTA and counts what it receives on one of two barriers,
by the round's parity, like an mbarrier: a phase ends when the CTA itself has arrived and all S
maps have come.  The scheduler delivers maps late and in any order, and lets any wait for
an incomplete round run out.  Whatever it does, no map may be on its way to a CTA that has left,
no map may count for another round than its own, and all CTAs leave.  Without a time-out every
round is received in full.  Two faulty protocols are caught: sending on after a time-out, and leaving
without the last round's settlement.
"""

import random

import pytest


class Fault(Exception):
    pass


class Cta:
    def __init__(self):
        self.phase = [0, 0]              # completed phases of each barrier
        self.arrived = [False, False]
        self.come = [0, 0]
        self.abort = False
        self.failed = False
        self.left = False
        self.sent = 0
        self.received = 0


class Cluster:
    def __init__(self, rng, size, rounds, patience, delivery=0.5,
                 stop_after_abort=True, settle=True):
        self.rng, self.size, self.rounds, self.patience = rng, size, rounds, patience
        self.delivery = delivery
        self.stop_after_abort, self.settle = stop_after_abort, settle
        self.ctas = [Cta() for _ in range(size)]
        self.flying = []                                    # (destination, round)
        self.at_barrier = [0] * size                        # cluster barriers passed
        self.timed_out = False

    # ---- hardware ----
    def complete(self, c):
        for b in (0, 1):
            if c.arrived[b] and c.come[b] == self.size:
                c.phase[b] += 1
                c.arrived[b], c.come[b] = False, 0

    def deliver(self):
        dst, n = self.flying.pop(self.rng.randrange(len(self.flying)))
        c = self.ctas[dst]
        if c.left:
            raise Fault(f"a map of round {n} reaches CTA {dst} after it has left")
        if c.phase[n & 1] != n >> 1:
            raise Fault(f"a map of round {n} counts for phase {c.phase[n & 1]}")
        c.come[n & 1] += 1
        self.complete(c)

    def send_map(self, c, n):
        if c.arrived[n & 1]:
            raise Fault(f"second arrival in a phase, round {n}")
        c.arrived[n & 1] = True
        self.flying += [(q, n) for q in range(self.size)]
        self.complete(c)

    def done(self, c, n):
        return c.phase[n & 1] > n >> 1

    # ---- the kernel, one CTA; yields wherever another may run ----
    def run(self, rank):
        c = self.ctas[rank]
        for n in range(self.rounds):
            stop = c.abort
            yield
            if not (stop and self.stop_after_abort):
                c.sent = n + 1
                self.send_map(c, n)
            while not c.abort and not self.done(c, n):
                if self.rng.random() < self.patience:
                    c.abort = self.timed_out = True
                yield
            c.received += self.done(c, n)
        if c.abort:
            for q in self.ctas:
                q.failed = True
        yield from self.barrier(rank, 1)
        if c.failed and self.settle:
            yield from self.barrier(rank, 2)
            most = max(q.sent for q in self.ctas)
            if most - c.sent not in (0, 1):
                raise Fault("more than a round apart")
            if c.sent < most:
                self.send_map(c, most - 1)
            for n in range(max(most - 2, 0), most):
                while not self.done(c, n):                  # bounded in the kernel
                    yield
        c.left = True

    def barrier(self, rank, k):
        self.at_barrier[rank] = k
        while min(self.at_barrier) < k:
            yield

    def simulate(self):
        live = [self.run(q) for q in range(self.size)]
        for _ in range(200000):
            if self.flying and (not live or self.rng.random() < self.delivery):
                self.deliver()
                continue
            if not live:
                return
            g = self.rng.choice(live)
            try:
                next(g)
            except StopIteration:
                live.remove(g)
        raise Fault("the CTAs do not end")


@pytest.mark.parametrize("size", [2, 3, 4, 8, 16])
@pytest.mark.parametrize("patience", [0.0, 0.002, 0.05, 0.5])
@pytest.mark.parametrize("delivery", [0.5, 0.05])
def test_no_map_is_on_its_way_to_a_cta_that_left(size, patience, delivery):
    timed_out = 0
    for seed in range(60):
        c = Cluster(random.Random(seed), size, 1 + seed % 7, patience, delivery)
        c.simulate()
        timed_out += c.timed_out
        if not c.timed_out:
            assert all(q.received == c.rounds for q in c.ctas)
    assert (timed_out == 0) == (patience == 0.0)


@pytest.mark.parametrize("fault", [dict(stop_after_abort=False, settle=False),
                                   dict(stop_after_abort=False), dict(settle=False)])
def test_the_faulty_protocols_are_caught(fault):
    caught = 0
    for seed in range(60):
        try:
            Cluster(random.Random(seed), 4, 5, 0.05, 0.05, **fault).simulate()
        except Fault:
            caught += 1
    assert caught > 20
