"""A CPU model of the ring protocol of the decode attention (csrc/attn_paged.cu):
a producer (or two, one for K and one for V) that issues granule copies in order,
a few at a time, into a ring of slots, and key warps that take the granules in turn (granule i of a segment
portion by warp i mod KW; with several row tiles, one warp of each).  A portion's
tiles may be fewer than the CTA's: the warps are then shared out to those, and
the first tile's warp arrives for the missing ones.  Copies
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

    def arrive(self, tx=0, n=1):
        if self.pending < n:
            raise Broken("an arrival more than the phase expects")
        self.pending -= n
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


def run(portions, slots, warps, rtc, seed, guard=True, slow=0.1, group=4, producers=1):
    """portions: (granules, row tiles with rows)"""
    rnd = random.Random(seed)
    full, empty = [Bar(producers) for _ in range(slots)], [Bar(rtc) for _ in range(slots)]
    content, readers = [[None] * producers for _ in range(slots)], [0] * slots
    time, order, heap = 0, 0, []

    def at(dt, fn):
        nonlocal order
        order += 1
        heapq.heappush(heap, (time + dt, order, fn))

    def latency(base):
        return base * (20 if rnd.random() < slow else 1) * rnd.uniform(0.5, 1.5)

    def producer(which):
        i = 0
        for cnt, _ in portions:
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
                        content[s][which] = k
                        full[s].tx -= 1
                        full[s].check()
                    at(latency(60), land)
                yield latency(4)
            i += cnt

    arrived = [0] * len(portions)                # warps at each portion's end

    def consumer(warp):
        base = 0
        for pn, (cnt, live) in enumerate(portions):
            rt, kw, kws = warp % live, warp // live, warps // live
            for gi in range(kw, cnt if kw < kws else 0, kws):
                k = base + gi
                s, use = k % slots, k // slots
                if guard and use > 0:
                    while not empty[s].passed(use - 1):
                        yield 1
                while not full[s].passed(use):
                    yield 1
                if content[s] != [k] * producers:
                    raise Broken("another granule than the expected one")
                readers[s] += 1
                yield latency(40)
                if content[s] != [k] * producers:
                    raise Broken("a slot changed while it was read")
                readers[s] -= 1
                empty[s].arrive(n=rtc - live + 1 if rt == 0 else 1)
            base += cnt
            arrived[pn] += 1                     # the joining barrier of the segment
            while arrived[pn] < warps:
                yield 1

    roles = [producer(i) for i in range(producers)] + [consumer(w) for w in range(warps)]
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


def portions_of(rnd, rtc):
    return [(rnd.choice([1, 3, 7, 17, 40, 70]), rnd.randint(1, rtc))
            for _ in range(rnd.randint(1, 4))]


@pytest.mark.parametrize("slots,warps,rtc,group,producers", [
    (12, 7, 1, 4, 1), (11, 7, 1, 2, 1), (23, 7, 1, 2, 1), (24, 7, 1, 4, 1), (6, 6, 1, 4, 1),
    (10, 10, 1, 2, 1), (10, 10, 2, 2, 2), (10, 10, 3, 4, 2), (13, 7, 2, 4, 1), (11, 7, 3, 4, 1),
    (14, 10, 3, 4, 2), (14, 10, 2, 4, 2)])
def test_ring(slots, warps, rtc, group, producers):
    for seed in range(25):
        run(portions_of(random.Random(seed), rtc), slots, warps, rtc, seed, group=group,
            producers=producers)


def test_a_wait_for_the_copy_alone_is_caught():
    caught = 0
    for seed in range(40):
        try:
            run([(200, 1)], 24, 15, 1, seed, guard=False, slow=0.2)
        except Broken:
            caught += 1
    assert caught > 0
