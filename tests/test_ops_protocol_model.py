"""Models of the attention and decay kernels' mbarrier handshakes, checked over random
interleavings (CPU).

Each role of a kernel (the TMA producer, the warp that issues the products, two
stand-ins for the compute threads, the storing thread) is an actor that runs a
few steps at a time in random order and at random speeds; the tensor cores and
the copy engine complete what was issued, in order, at times of their own.  The
barriers keep the hardware's parity semantics: a parity wait passes while the
current phase's parity differs from the one asked for, so a waiter that two
phases have passed by waits for ever.  Checked: nothing deadlocks; no tile is
read before it has landed or refilled (or staged over) before its readers are
done; accumulators are read and overwritten in the right order.

The variants with one barrier for the score products of even and odd key tiles
(dQ), and for the staged output tiles (decay walk), must fail: a late waiter
misses a phase there.
"""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase, self.tx = count, count, 0, 0

    def arrive(self, tx=0):
        self.pending -= 1
        self.tx += tx
        assert self.pending >= 0, "more arrivals than the count in one phase"
        self._maybe()

    def complete(self, tx):
        self.tx -= tx
        self._maybe()

    def _maybe(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, phase):
        return (self.phase & 1) != (phase & 1)


def wait(bar, phase):
    while not bar.done(phase):
        yield


class Machine:
    """Actors, an in-order tensor pipe and an in-order copy engine."""

    def __init__(self, seed, limit=60000):
        self.rnd, self.limit = random.Random(seed), limit
        self.actors, self.speed, self.pipe, self.copies = [], [], [], []

    def add(self, gen):
        self.actors.append(gen)
        self.speed.append(self.rnd.choice([1.0, 0.3, 0.05]))

    def mma(self, *fns):          # executed when the products before it are done
        self.pipe.extend(fns)

    def copy(self, fn):
        self.copies.append(fn)

    def run(self):
        alive, quiet = list(range(len(self.actors))), 0
        for _ in range(self.limit):
            if not alive:
                assert not self.pipe and not self.copies, "work in flight at the end"
                return
            for q, p in ((self.pipe, 0.4), (self.copies, 0.2)):
                if q and self.rnd.random() < p:
                    q.pop(0)()
            i = self.rnd.choice(alive)
            if self.rnd.random() < self.speed[i]:
                try:
                    next(self.actors[i])
                except StopIteration:
                    alive.remove(i)
        raise AssertionError("deadlock")


class Ring:
    def __init__(self, m, slots, tiles):
        self.m, self.slots, self.tiles = m, slots, tiles
        self.full = [Bar(1) for _ in range(slots)]
        self.empty = [Bar(1) for _ in range(slots)]
        self.holds, self.users = [None] * slots, [0] * slots

    def producer(self):
        for t in range(self.tiles):
            k = t % self.slots
            if t >= self.slots:
                yield from wait(self.empty[k], t // self.slots - 1)
            assert self.users[k] == 0, "refilled while in use"
            self.holds[k] = None
            self.full[k].arrive(tx=1)

            def land(k=k, t=t):
                self.holds[k] = t
                self.full[k].complete(1)
            self.m.copy(land)
            yield
        for t in range(max(0, self.tiles - self.slots), self.tiles):
            yield from wait(self.full[t % self.slots], t // self.slots)

    def arrived(self, t):
        yield from wait(self.full[t % self.slots], t // self.slots)

    def use(self, t):              # a product that reads tile t: now until it has run
        k = t % self.slots
        assert self.holds[k] == t, "read before it landed"
        self.users[k] += 1

        def over(k=k):
            self.users[k] -= 1
        return over

    def release(self, t):
        if t + self.slots < self.tiles:
            self.m.mma(self.empty[t % self.slots].arrive)


def dq_model(n, seed, barriers=2):
    m = Machine(seed)
    r = Ring(m, 5, 2 * n)
    barS, barD, barDs, end = [Bar(1) for _ in range(barriers)], Bar(1), Bar(2), Bar(1)
    S, P = [None, None], [None]           # which tile's scores the accumulators hold
    phase = (lambda i: (barS[i & 1], i >> 1)) if barriers == 2 else (lambda i: (barS[0], i))

    def product(t, bar, put):
        over = r.use(t)
        m.mma(over, put)
        if bar is not None:
            m.mma(bar.arrive)

    def issue():
        def scores(i):
            yield from r.arrived(2 * i)
            product(2 * i, phase(i)[0], lambda: S.__setitem__(i & 1, i))

        def dscores(i):
            yield from r.arrived(2 * i + 1)
            product(2 * i + 1, None, lambda: P.__setitem__(0, i))
            r.release(2 * i + 1)
            m.mma(barD.arrive)
        yield from scores(0)
        yield from dscores(0)
        for i in range(n):
            if i + 1 < n:
                yield from scores(i + 1)
            yield from wait(barDs, i)
            product(2 * i, None, lambda: None)
            r.release(2 * i)
            if i + 1 < n:
                yield from dscores(i + 1)
            yield
        m.mma(end.arrive)

    def compute():
        for i in range(n):
            yield from wait(*phase(i))
            assert S[i & 1] == i, "scores of another tile"
            yield
            yield from wait(barD, i)
            assert P[0] == i, "dP of another tile"
            yield
            barDs.arrive()
            yield
        yield from wait(end, 0)

    for a in (r.producer(), issue(), compute(), compute()):
        m.add(a)
    m.run()


def dkv_model(n, seed):
    m = Machine(seed)
    r = Ring(m, 4, 2 * n)
    barS, barD, barP, barDs, end = Bar(1), Bar(1), Bar(2), Bar(2), Bar(1)
    S, P = [None], [None]

    def product(t, put, bar=None):
        m.mma(r.use(t), put)
        if bar is not None:
            m.mma(bar.arrive)

    def issue():
        def scores(i):
            yield from r.arrived(2 * i)
            product(2 * i, lambda: S.__setitem__(0, i), barS)

        def dscores(i):
            yield from r.arrived(2 * i + 1)
            product(2 * i + 1, lambda: P.__setitem__(0, i), barD)
        yield from scores(0)
        yield from dscores(0)
        for i in range(n):
            yield from wait(barP, i)
            product(2 * i + 1, lambda: None)
            if i + 1 < n:
                yield from scores(i + 1)
            yield from wait(barDs, i)
            product(2 * i, lambda: None)
            r.release(2 * i)
            r.release(2 * i + 1)
            if i + 1 < n:
                yield from dscores(i + 1)
        m.mma(end.arrive)

    def compute():
        for i in range(n):
            yield from wait(barS, i)
            assert S[0] == i
            yield
            barP.arrive()
            yield from wait(barD, i)
            assert P[0] == i
            yield
            barDs.arrive()
        yield from wait(end, 0)

    for a in (r.producer(), issue(), compute(), compute()):
        m.add(a)
    m.run()


def fwd_model(n0, n1, seed, dual=False):
    """Two query tiles of n0 and n1 key tiles, or one whose key tiles alternate (dual, n0 in all)."""
    m = Machine(seed)
    total = max(n0, n1)
    n = [(total + 1) // 2, total // 2] if dual else [n0, n1]
    r = Ring(m, 5, 2 * total)
    barS, barO = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
    barP = [[Bar(2), Bar(2)], [Bar(2), Bar(2)]]
    S, O = [None, None], [0, 0]

    def issue():
        def scores(x, i, j):
            m.mma(r.use(2 * i), lambda: S.__setitem__(x, j), barS[x].arrive)

        def values(x, i, j):
            for h in range(2):
                yield from wait(barP[x][h], j)
                m.mma(r.use(2 * i + 1))
            m.mma(lambda: O.__setitem__(x, j + 1))
            if j + 1 == n[x]:
                m.mma(barO[x].arrive)
        yield from r.arrived(0)
        if dual:
            scores(0, 0, 0)
            r.release(0)
            if total > 1:
                yield from r.arrived(2)
                scores(1, 1, 0)
                r.release(2)
            for i in range(total):
                yield from r.arrived(2 * i + 1)
                yield from values(i & 1, i, i >> 1)
                r.release(2 * i + 1)
                if i + 2 < total:
                    yield from r.arrived(2 * i + 4)
                    scores(i & 1, i + 2, (i >> 1) + 1)
                    r.release(2 * i + 4)
            return
        for x in range(2):
            if n[x]:
                scores(x, 0, 0)
        r.release(0)
        for i in range(total):
            yield from r.arrived(2 * i + 1)
            if i + 1 < total:
                yield from r.arrived(2 * i + 2)
            for x in range(2):
                if i < n[x]:
                    yield from values(x, i, i)
                if x == 1:
                    r.release(2 * i + 1)
                if i + 1 < n[x]:
                    scores(x, i + 1, i + 1)
            if i + 1 < total:
                r.release(2 * i + 2)

    def compute(x):
        for i in range(n[x]):
            tile = 2 * i + x if dual else i
            yield from r.arrived(2 * tile + 1)      # (a ragged V tile's rows are cleared)
            yield from wait(barS[x], i)
            assert S[x] == i and O[x] == i, "O rescaled beside its product"
            for h in range(2):
                yield
                barP[x][h].arrive()
        if n[x]:
            yield from wait(barO[x], 0)

    for a in [r.producer(), issue()] + [compute(x) for x in (0, 0, 1, 1)]:
        m.add(a)
    m.run()


def walk_model(n, seed, stores=2):
    """The decay walk: tiles a, b, c of n chunks; masks and output by one group, state and
    scaling by another, staged output tiles over c by a storing thread."""
    m = Machine(seed)
    r = Ring(m, 5, 3 * n)
    barP, barX, barO = Bar(1), Bar(1), Bar(1)
    barPm, barS, barOf = Bar(2), Bar(2), Bar(2)
    barK, barSt = [Bar(2), Bar(2)], [Bar(2) for _ in range(stores)]
    P, O, X = [None], [None], [None]
    st = (lambda i: (barSt[i & 1], i >> 1)) if stores == 2 else (lambda i: (barSt[0], i))

    def issue():
        def scores(i):
            yield from r.arrived(3 * i)
            yield from r.arrived(3 * i + 1)
            m.mma(r.use(3 * i), r.use(3 * i + 1), lambda: P.__setitem__(0, i), barP.arrive)
        yield from scores(0)
        for i in range(n):
            yield from wait(barS, i)
            if i:
                yield from wait(barOf, i - 1)
            m.mma(r.use(3 * i))
            r.release(3 * i)
            yield from r.arrived(3 * i + 2)
            for h in range(2):
                yield from wait(barK[h], i)
                m.mma(r.use(3 * i + 1), r.use(3 * i + 2))
            m.mma(lambda i=i: X.__setitem__(0, i), barX.arrive)
            r.release(3 * i + 1)
            yield from wait(barPm, i)
            m.mma(r.use(3 * i + 2), lambda i=i: O.__setitem__(0, i), barO.arrive)
            if i + 1 < n:
                yield from scores(i + 1)

    def masks():
        def output(i):
            yield from wait(barO, i)
            assert O[0] == i
            yield
            barOf.arrive()
            k = (3 * i + 2) % 5
            assert r.holds[k] == 3 * i + 2 and r.users[k] == 0, "staged over a tile in use"
            yield
            st(i)[0].arrive()
        for i in range(n):
            if i:
                yield from output(i - 1)
            yield from wait(barP, i)
            assert P[0] == i
            yield
            barPm.arrive()
        yield from output(n - 1)

    def state():
        for i in range(n):
            if i:
                yield from wait(barX, i - 1)
                assert X[0] == i - 1
            yield
            barS.arrive()
            yield from r.arrived(3 * i + 1)
            yield from wait(barP, i)
            for h in range(2):
                yield
                barK[h].arrive()

    def store():
        for i in range(n):
            yield from wait(*st(i))
            for _ in range(m.rnd.choice([1, 1, 40])):   # the store reads the tile
                yield
            if 3 * i + 2 + 5 < 3 * n:
                r.empty[(3 * i + 2) % 5].arrive()

    for a in (r.producer(), issue(), masks(), masks(), state(), state(), store()):
        m.add(a)
    m.run()


@pytest.mark.parametrize("n", [1, 2, 3, 4, 7])
def test_handshakes_hold(n):
    for seed in range(60):
        dq_model(n, seed)
        dkv_model(n, seed)
        walk_model(n, seed)
        fwd_model(n, n + seed % 2, seed)
        fwd_model(n, n, seed, dual=True)
    fwd_model(0, n, 0)                     # a first tile whose rows see no key


def fails(model, *args, **kw):
    failed = 0
    for seed in range(150):
        try:
            model(*args, seed, **kw)
        except AssertionError:
            failed += 1
    return failed


def test_one_barrier_for_the_scores_of_both_buffers_fails():
    assert fails(dq_model, 5, barriers=1) > 0


def test_one_barrier_for_the_staged_tiles_fails():
    assert fails(walk_model, 9, stores=1) > 0
