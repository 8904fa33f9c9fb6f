"""A CPU model of the ring protocol of the decode attention (csrc/attn_paged.cu):
one producer that issues granule copies in order, a few at a time, into a ring
of slots, and key warps that take the granules in turn (granule i of a segment
portion by warp i mod KW; with several row tiles, one warp of each).  Copies
land and warps work for random times, and mbarrier waits have the hardware's
parity semantics.

Checked over random portions: every warp reads the granule it expects, no slot
is written while it is read or before it was read, every wait is for the phase
it means, every barrier gets exactly its arrivals, nothing deadlocks.  The
variant in which a warp waits for its copy without first waiting for the
slot's previous granule to have been taken must be caught: with slots not a
multiple of the key warps, the previous granule belongs to another warp, and
its copy may land later.
"""
import heapq
import random

import pytest


class Broken(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.tx, self.n = count, count, 0, 0

    def arrive(self, tx=0):
        if self.pending == 0:
            raise Broken("an arrival more than the phase expects")
        self.pending -= 1
        self.tx += tx
        self.check()

    def check(self):
        if self.pending == 0 and self.tx == 0:
            self.n += 1
            self.pending = self.count

    def passed(self, phase, strict=True):
        """The parity wait for `phase`; raises where it passes for another one."""
        ok = (self.n & 1) != (phase & 1)
        if ok and strict and self.n <= phase:
            raise Broken("a wait passed before its phase")
        return ok


def run(portions, slots, kws, rtc, seed, guard=True, slow=0.1, group=4):
    rnd = random.Random(seed)
    full, empty = [Bar(1) for _ in range(slots)], [Bar(rtc) for _ in range(slots)]
    content, readers = [None] * slots, [0] * slots
    time, order, heap = 0, 0, []

    def at(dt, fn):
        nonlocal order
        order += 1
        heapq.heappush(heap, (time + dt, order, fn))

    def latency(base):
        return base * (20 if rnd.random() < slow else 1) * rnd.uniform(0.5, 1.5)

    def producer():
        i = 0
        for cnt in portions:
            for b in range(0, cnt, group):
                batch = range(i + b, i + min(b + group, cnt))
                for k in batch:
                    phase = k // slots - 1
                    while phase >= 0 and not empty[k % slots].passed(phase):
                        yield 1
                for k in batch:
                    s = k % slots
                    if readers[s]:
                        raise Broken("a slot is written while it is read")
                    full[s].arrive(tx=1)

                    def land(k=k, s=s):
                        content[s] = k
                        full[s].tx -= 1
                        full[s].check()
                    at(latency(60), land)
                yield latency(4)
            i += cnt

    arrived = [0] * len(portions)                # warps at each portion's end

    def consumer(kw):
        base = 0
        for pn, cnt in enumerate(portions):
            for gi in range(kw, cnt, kws):
                k = base + gi
                s, use = k % slots, k // slots
                if guard and use > 0:
                    while not empty[s].passed(use - 1):
                        yield 1
                while not full[s].passed(use):
                    yield 1
                if content[s] != k:
                    raise Broken("another granule than the expected one")
                readers[s] += 1
                yield latency(40)
                if content[s] != k:
                    raise Broken("a slot changed while it was read")
                readers[s] -= 1
                empty[s].arrive()
            base += cnt
            arrived[pn] += 1                     # the joining barrier of the segment
            while arrived[pn] < kws * rtc:
                yield 1

    roles = [producer()] + [consumer(kw) for kw in range(kws) for _ in range(rtc)]
    alive = len(roles)

    def step(r):
        nonlocal alive
        try:
            dt = next(r)
        except StopIteration:
            alive -= 1
            return
        at(dt, lambda: step(r))

    for r in roles:
        at(rnd.random(), lambda r=r: step(r))
    while heap and alive:
        time, _, fn = heapq.heappop(heap)
        if time > 1e6:
            raise Broken("deadlock")
        fn()
    if alive:
        raise Broken("deadlock")


def portions_of(rnd):
    return [rnd.choice([1, 3, 7, 17, 40, 70]) for _ in range(rnd.randint(1, 4))]


@pytest.mark.parametrize("slots,kws,rtc,group", [
    (12, 7, 1, 4), (11, 7, 1, 2), (23, 7, 1, 2), (24, 7, 1, 4), (6, 6, 1, 4), (10, 10, 1, 2),
    (10, 5, 2, 2), (10, 3, 3, 4), (13, 3, 2, 4)])
def test_ring(slots, kws, rtc, group):
    for seed in range(25):
        run(portions_of(random.Random(seed)), slots, kws, rtc, seed, group=group)


def test_a_wait_for_the_copy_alone_is_caught():
    caught = 0
    for seed in range(40):
        try:
            run([200], 24, 15, 1, seed, guard=False, slow=0.2)
        except Broken:
            caught += 1
    assert caught > 0
