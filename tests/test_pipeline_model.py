"""A discrete model of the two-issuer forward pipeline's barriers, run with random latencies.

Modelled as attn_fwd_kernel.cuh has them: the producer's three slots for K and V tiles in turn,
the S issuer, the PV issuer, the softmax groups, and mbarriers whose parity wait passes when the
barrier's current phase has the other parity.  A product that reads a slot not holding its tile,
a load into a slot being read, an arrival on a barrier that expects none, a pipeline that stops
and an exit with loads in flight are faults.

With one full barrier per slot, shared by the slot's K and V loads, each issuer sees every other
phase and its wait can pass two phases early; with a barrier for each kind it cannot.
"""
import heapq
import random

import pytest

SLOTS = 3


class Fault(Exception):
    pass


class Barrier:
    def __init__(self):
        self.pending, self.tx, self.phase = 1, 0, 0

    def _settle(self):
        if self.pending == 0 and self.tx == 0:
            self.phase, self.pending = self.phase + 1, 1

    def arrive(self, tx=0):
        if self.pending == 0:
            raise Fault("an arrival too many")
        self.tx += tx
        self.pending -= 1
        self._settle()

    def complete(self, tx):
        self.tx -= tx
        self._settle()

    def passes(self, parity):
        return (self.phase & 1) != parity


def run(T, groups, split, latency, rng):
    events, now, order, tensor_pipe = [], 0.0, 0, 0.0
    k_full, v_full = ([Barrier() for _ in range(SLOTS)] for _ in range(2))
    if not split:
        v_full = k_full
    empty = [Barrier() for _ in range(SLOTS)]
    s_full, s_free, p_full, pv_done = ([Barrier() for _ in range(2)] for _ in range(4))
    held, readers, flying = [None] * SLOTS, [0] * SLOTS, set()

    def at(delay, f):
        nonlocal order
        order += 1
        heapq.heappush(events, (now + delay, order, f))

    loads = [("K", 0)] + [x for t in range(T) for x in ((("K", t + 1),) if t + 1 < T else ()) + (("V", t),)]
    index = {x: i for i, x in enumerate(loads)}

    def product(slot, tile, done):
        nonlocal tensor_pipe
        if held[slot] != tile:
            raise Fault("a product reads a tile that is not there")
        readers[slot] += 1
        tensor_pipe = max(now, tensor_pipe) + 0.15

        def finished():
            readers[slot] -= 1
            for b in done:
                b.arrive()
        at(tensor_pipe + 0.3 - now, finished)

    def producer():
        for i, tile in enumerate(loads):
            slot = i % SLOTS
            if i >= SLOTS:
                yield lambda: empty[slot].passes((i // SLOTS - 1) & 1)
            if readers[slot]:
                raise Fault("a load into a slot being read")
            full = (k_full if tile[0] == "K" else v_full)[slot]
            full.arrive(1)
            held[slot] = None
            flying.add(i)

            def landed(i=i, slot=slot, tile=tile, full=full):
                flying.discard(i)
                held[slot] = tile
                full.complete(1)
            at(latency(rng), landed)

    def issuer(kind, full, wait_for, done):
        parity = [0] * SLOTS
        for t in range(T):
            i = index[(kind, t)]
            slot = i % SLOTS
            p = parity[slot] if split else (i // SLOTS) & 1
            parity[slot] ^= 1
            yield lambda: full[slot].passes(p)
            for g in range(groups):
                if kind == "V" or t > 0:
                    yield lambda: wait_for[g].passes((t if kind == "V" else t - 1) & 1)
                product(slot, (kind, t), [done[g]] + ([empty[slot]] if g == groups - 1 else []))

    def softmax(g):
        for t in range(T):
            yield lambda: s_full[g].passes(t & 1)
            yield rng.uniform(0.1, 0.6)
            s_free[g].arrive()
            if t:
                yield lambda: pv_done[g].passes((t - 1) & 1)
            yield rng.uniform(0.05, 0.2)
            p_full[g].arrive()
        yield lambda: pv_done[g].passes((T - 1) & 1)

    roles = [producer(), issuer("K", k_full, s_free, s_full), issuer("V", v_full, p_full, pv_done)]
    roles += [softmax(g) for g in range(groups)]
    waiting, running = {}, set(range(len(roles)))

    def step(r):
        while True:
            try:
                w = next(roles[r])
            except StopIteration:
                running.discard(r)
                return
            if not callable(w):
                at(w, lambda: step(r))
                return
            if not w():
                waiting[r] = w
                return

    for r in list(running):
        step(r)
    while events:
        now, _, f = heapq.heappop(events)
        f()
        ready = True
        while ready:
            ready = [r for r in waiting if waiting[r]()]
            for r in ready:
                del waiting[r]
                step(r)
    if running:
        raise Fault("the pipeline stops")
    if flying:
        raise Fault("an exit with loads in flight")


LATENCIES = [lambda r: r.uniform(0.8, 1.0), lambda r: r.uniform(0.8, 3.0),
             lambda r: r.uniform(0.8, 1.2) + (r.random() < 0.1) * r.uniform(0, 6)]


@pytest.mark.parametrize("groups", [1, 2])
def test_a_barrier_for_each_kind_of_load(groups):
    for latency in LATENCIES:
        for seed in range(300):
            rng = random.Random(seed)
            run(rng.randint(1, 14), groups, True, latency, rng)


def test_a_shared_barrier_fails():
    with pytest.raises(Fault):
        for seed in range(300):
            rng = random.Random(seed)
            run(rng.randint(1, 14), 2, False, LATENCIES[1], rng)
