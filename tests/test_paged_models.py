"""Models of the kernels over pages (CPU): how the keys are cut into runs, and the handshakes of
the warps over random interleavings, on the machine of the other kernels' models but for copies,
which land in any order here."""
import random

import pytest

from test_ops_protocol_model import Bar, Machine, wait

KEYS = 128


# ---- runs ---------------------------------------------------------------------------------
def items(ql, kl, S, extra):
    """(keys, width) of a sequence's items."""
    n = -(-ql // S)
    keys = [kl if i + 1 == n else max(0, kl - ql + (i + 1) * S) for i in range(n)]
    return [(k, extra + k) for k in keys]


def before(ql, kl, S, i, extra):
    """The kernel's closed form of the widths of the first i items."""
    n, off = -(-ql // S), kl - ql
    flat = 0 if off >= 0 else min(n - 1, -off // S)
    return i * extra + (0 if i <= flat else (i - flat) * off + S * ((flat + 1 + i) * (i - flat) // 2))


def test_widths_in_closed_form():
    rnd = random.Random(1)
    for _ in range(5000):
        S, extra = rnd.choice([256, 128, 84, 64, 50, 42, 32, 2]), rnd.choice([128, 512])
        ql, kl = rnd.randint(1, 3000), rnd.choice([0, rnd.randint(0, 100), rnd.randint(0, 5000)])
        at = 0
        for i, (_, wide) in enumerate(items(ql, kl, S, extra)):
            assert before(ql, kl, S, i, extra) == at
            at += wide


def tiles(x, wide, extra):
    return -(-(wide - extra) // KEYS) if x >= wide else max(0, x - extra) // KEYS


def test_every_key_tile_is_one_run_s():
    """Each tile of each item once; an item is either one run's alone or joined from parts of consecutive
    runs, the first of them in the slot for items that begin in their run."""
    rnd = random.Random(2)
    for _ in range(1000):
        S, Hk, extra = rnd.choice([256, 84, 64, 32, 2]), rnd.choice([1, 2, 3]), rnd.choice([128, 512])
        most, narrow = rnd.choice([1, 2, 5, 28, 152, 304]), rnd.choice([1, 256, 768])
        seqs = [(rnd.choice([0, 1, 1, 1, rnd.randint(1, 600)]), rnd.choice([0, rnd.randint(0, 3000)])) for _ in range(rnd.randint(1, 8))]
        all_of = [it for q, k in seqs for _ in range(Hk) for it in items(q, k, S, extra)]
        V = sum(w for _, w in all_of)
        C = most if V >= narrow * most else max(1, V // narrow)
        begin = lambda c: V // C * c + min(c, V % C)
        pos = 0
        for keys, wide in all_of:
            n, owners, got, parts, join = -(-keys // KEYS), [], [], [], None
            for c in range(C):
                lo, hi = max(begin(c), pos), min(begin(c + 1), pos + wide)
                if lo >= hi:
                    continue
                x0, x1 = lo - pos, hi - pos
                a, b, whole, mine = tiles(x0, wide, extra), tiles(x1, wide, extra), True, True
                if x0 > 0 or x1 < wide:
                    begins = (begin(c) if x0 > 0 else begin(c + 1) - x1 + x0) - x0
                    last = c
                    while last + 1 < C and begin(last + 1) < begins + wide:
                        last += 1
                    whole = tiles(max(0, begin(last) - begins), wide, extra) == 0
                    mine = not whole or last == c
                    if mine and not whole and x0 == 0:
                        join = (c, last)
                if not mine:
                    assert a == b
                    continue
                (owners if whole else parts).append((c, x0 > 0))
                got += range(a, b)
            assert got == list(range(n))
            if owners:
                assert len(owners) == 1 and not parts and join is None
            else:
                assert [c for c, _ in parts] == list(range(join[0], join[1] + 1))
                assert [first for _, first in parts] == [False] + [True] * (len(parts) - 1)
            pos += wide


def test_division_by_multiplication():
    """Page of a row: (umulhi(mul, row) + row) >> shift for rows below 2^31 and any page size."""
    rnd = random.Random(3)
    for page in list(range(16, 600, 16)) + [4096, 65520, 1 << 20, (1 << 20) + 16, 1 << 30]:
        shift = 0
        while 1 << shift < page:
            shift += 1
        mul = (((1 << shift) - page << 32) // page + 1) & 0xffffffff
        near = [k * page + d for k in (rnd.randrange((1 << 31) // page) for _ in range(50)) for d in (-1, 0, 1)]
        for row in near + [0, (1 << 31) - 1] + [rnd.randrange(1 << 31) for _ in range(50)]:
            if row >= 0:
                assert (mul * row >> 32) + row >> shift == row // page


# ---- handshakes -----------------------------------------------------------------------------
class Loose(Machine):
    """Copies land in any order, some of them late."""

    def copy(self, fn):
        late = [self.rnd.choice([0] * 9 + [60])]

        def land():
            if late[0]:
                late[0] -= 1
                self.copies.append(land)
            else:
                fn()
        self.copies.insert(self.rnd.randint(0, len(self.copies)), land)


class Ring:
    """A ring of slots that goes on over items."""

    def __init__(self, m, slots):
        self.m, self.slots = m, slots
        self.full, self.empty = ([Bar(1) for _ in range(slots)] for _ in range(2))
        self.holds, self.users = [None] * slots, [0] * slots

    def load(self, t):
        k = t % self.slots
        if t >= self.slots:
            yield from wait(self.empty[k], t // self.slots - 1)
        assert self.users[k] == 0, "refilled while in use"
        self.holds[k] = None
        self.full[k].arrive(tx=1)

        def land():
            self.holds[k] = t
            self.full[k].complete(1)
        self.m.copy(land)
        yield

    def landed(self, t):
        yield from wait(self.full[t % self.slots], t // self.slots)

    def use(self, t):
        k = t % self.slots
        assert self.holds[k] == t, "read before it landed"
        self.users[k] += 1

        def over():
            self.users[k] -= 1
        return over

    def release(self, t):
        self.m.mma(self.empty[t % self.slots].arrive)

    def end(self, t):
        for u in range(max(0, t - self.slots), t):
            yield from wait(self.empty[u % self.slots], u // self.slots)


def meet(bar, phases, me):
    """A barrier of several actors."""
    bar.arrive()
    yield from wait(bar, phases[me])
    phases[me] += 1


def many_model(work, seed, clear_ahead=False):
    """k_paged_many over items (tiles of group 0, of group 1, dual).  clear_ahead: rows past the keys
    cleared before S is waited for."""
    m = Loose(seed)
    r = Ring(m, 4)
    barQ, barQF, barS, barO = ([Bar(1), Bar(1)] for _ in range(4))
    barP, barF = [[Bar(2), Bar(2)] for _ in range(2)], [Bar(2), Bar(2)]
    Q, Qusers, S, O = [None, None], [0, 0], [None, None], [None, None]
    pair, phases = Bar(4), [0] * 4
    loaded = lambda n: n[0] + n[1] if n[2] else max(n[0], n[1])

    def loads():
        t, qc = 0, [0, 0]
        for e, n in enumerate(work):
            for i in range(loaded(n)):
                for _ in "kv":
                    yield from r.load(t)
                    t += 1
                if i:
                    continue
                for x in range(2):
                    if n[x] and not (n[2] and x):
                        if qc[x]:
                            yield from wait(barQF[x], qc[x] - 1)
                        assert not Qusers[x], "queries replaced while in use"
                        Q[x] = None
                        barQ[x].arrive(tx=1)

                        def land(x=x, e=e):
                            Q[x] = e
                            barQ[x].complete(1)
                        m.copy(land)
                        qc[x] += 1
                        yield
        for u in range(max(0, t - r.slots), t):
            yield from r.landed(u)

    def issues():
        t0, qc, oc, sc = 0, [0, 0], [0, 0], [0, 0]
        for e, n in enumerate(work):
            k = loaded(n)
            if not k:
                continue

            def scores(x, q, i, last):
                assert Q[q] == e, "other queries"
                over = r.use(t0 + 2 * i)
                Qusers[q] += 1

                def done(e=e):
                    over()
                    Qusers[q] -= 1
                    S[x] = ("S", e, i)
                m.mma(done, barS[x].arrive)
                if last:
                    m.mma(barQF[q].arrive)

            def values(x, i, j):
                if j == 0 and oc[x]:
                    yield from wait(barF[x], oc[x] - 1)
                for h in range(2):
                    yield from wait(barP[x][h], sc[x] + j)

                def done(over=r.use(t0 + 2 * i + 1), e=e):
                    over()
                    assert S[x] == ("P", e, i), "no P there"
                    assert j == 0 or O[x] == (e, j), "O of something else"
                    O[x] = (e, j + 1)
                m.mma(done)
                if j + 1 == n[x]:
                    m.mma(barO[x].arrive)
            yield from r.landed(t0)
            if n[0]:
                yield from wait(barQ[0], qc[0])
            if n[2]:
                scores(0, 0, 0, k == 1)
                r.release(t0)
                if k > 1:
                    yield from r.landed(t0 + 2)
                    scores(1, 0, 1, k == 2)
                    r.release(t0 + 2)
                for i in range(k):
                    yield from r.landed(t0 + 2 * i + 1)
                    yield from values(i & 1, i, i >> 1)
                    r.release(t0 + 2 * i + 1)
                    if i + 2 < k:
                        yield from r.landed(t0 + 2 * i + 4)
                        scores(i & 1, 0, i + 2, i + 3 == k)
                        r.release(t0 + 2 * i + 4)
                qc[0] += 1
            else:
                if n[0]:
                    scores(0, 0, 0, n[0] == 1)
                if n[1]:
                    yield from wait(barQ[1], qc[1])
                    scores(1, 1, 0, n[1] == 1)
                r.release(t0)
                for i in range(k):
                    yield from r.landed(t0 + 2 * i + 1)
                    if i + 1 < k:
                        yield from r.landed(t0 + 2 * i + 2)
                    for x in range(2):
                        if i < n[x]:
                            yield from values(x, i, i)
                        if x == 1:
                            r.release(t0 + 2 * i + 1)
                        if i + 1 < n[x]:
                            scores(x, x, i + 1, i + 2 == n[x])
                    if i + 1 < k:
                        r.release(t0 + 2 * i + 2)
                qc[0] += n[0] > 0
                qc[1] += n[1] > 0
            t0 += 2 * k
            for x in range(2):
                oc[x] += n[x] > 0
                sc[x] += n[x]
            yield
        yield from r.end(t0)
        for x in range(2):
            if qc[x]:
                yield from wait(barQF[x], qc[x] - 1)

    def softmax(x, me):
        t0, s0, done = 0, 0, 0
        for e, n in enumerate(work):
            k = loaded(n)
            for j in range(n[x]):
                i = 2 * j + x if n[2] else j
                tail, t = i + 1 == k, t0 + 2 * i + 1

                def clear():
                    yield from r.landed(t)
                    assert r.holds[t % r.slots] == t, "rows of another tile cleared"
                    yield
                if tail and clear_ahead:
                    yield from clear()
                yield from wait(barS[x], s0 + j)
                assert S[x] in (("S", e, i), ("P", e, i)), "scores of another tile"
                if tail and not clear_ahead:
                    yield from clear()
                yield
                assert j == 0 or O[x] == (e, j), "O not idle"
                for h in range(2):
                    if barP[x][h].pending == 1:     # the second of the two stand-ins: P is whole
                        S[x] = ("P", e, i)
                    barP[x][h].arrive()
                    yield
            t0 += 2 * k
            s0 += n[x]
            if n[x]:
                yield from wait(barO[x], done)
                assert O[x] == (e, n[x]), "not this item's output"
                done += 1
            if n[2]:
                for _ in range(2):
                    yield from meet(pair, phases, me)
            yield
            if n[x]:
                assert O[x] == (e, n[x]), "output overwritten"
                barF[x].arrive()
    actors = [loads(), issues()] + [softmax(x, 2 * x + i) for x in range(2) for i in range(2)]
    for a in actors:
        m.add(a)
    m.run()


def some_work(seed):
    rnd = random.Random(seed)
    work = []
    for _ in range(rnd.randint(1, 7)):
        if rnd.random() < 0.4:
            k = rnd.randint(0, 5)
            work.append((k - k // 2, k // 2, True))
        else:
            n = rnd.choice([(1, 1), (0, 2), (0, 0), (3, 4), (1, 5), (2, 2), (4, 0)])
            work.append((*n, False))
    return work


def fails(model, n=60):
    failed = 0
    for seed in range(n):
        try:
            model(seed)
        except AssertionError:
            failed += 1
    return failed


def test_two_query_tiles_over_items():
    for seed in range(250):
        many_model(some_work(seed), seed)


def test_rows_cleared_ahead_of_the_scores_fail():
    """A group whose part of an item was short is rounds of the ring ahead."""
    assert fails(lambda seed: many_model([(1, 6, False), (1, 1, False), (1, 4, False), (1, 1, False)], seed, clear_ahead=True)) > 0


def few_model(work, seed):
    """k_paged_few over items of n key tiles."""
    m = Loose(seed)
    r = Ring(m, 4)
    barQ, barQF, barS, barO, barP, barF = Bar(1), Bar(1), Bar(1), Bar(1), Bar(2), Bar(2)
    Q, S, O = [None], [None], [None]

    def loads():
        t, qc = 0, 0
        for e, n in enumerate(work):
            for i in range(n):
                for _ in "kv":
                    yield from r.load(t)
                    t += 1
                if i == 0:
                    if qc:
                        yield from wait(barQF, qc - 1)
                    Q[0] = None
                    barQ.arrive(tx=1)

                    def land(e=e):
                        Q[0] = e
                        barQ.complete(1)
                    m.copy(land)
                    qc += 1
                    yield
        for u in range(max(0, t - r.slots), t):
            yield from r.landed(u)

    def issues():
        t0, qc, sc = 0, 0, 0
        for e, n in enumerate(work):
            if not n:
                continue

            def scores(i):
                yield from r.landed(t0 + 2 * i)
                assert Q[0] == e, "other queries"

                def done(over=r.use(t0 + 2 * i), e=e):
                    over()
                    S[0] = ("S", e, i)
                m.mma(done, barS.arrive)
                r.release(t0 + 2 * i)
                if i + 1 == n:
                    m.mma(barQF.arrive)
            yield from wait(barQ, qc)
            yield from scores(0)
            for i in range(n):
                yield from r.landed(t0 + 2 * i + 1)
                if i == 0 and qc:
                    yield from wait(barF, qc - 1)
                yield from wait(barP, sc + i)

                def done(over=r.use(t0 + 2 * i + 1), i=i, e=e):
                    over()
                    assert S[0] == ("P", e, i)
                    O[0] = (e, i + 1)
                m.mma(done)
                r.release(t0 + 2 * i + 1)
                if i + 1 < n:
                    yield from scores(i + 1)
                yield
            m.mma(barO.arrive)
            t0, sc, qc = t0 + 2 * n, sc + n, qc + 1
        yield from r.end(t0)
        if qc:
            yield from wait(barQF, qc - 1)

    def softmax():
        t0, s0, done = 0, 0, 0
        for e, n in enumerate(work):
            for i in range(n):
                if i + 1 == n:     # rows past the keys
                    yield from r.landed(t0 + 2 * i + 1)
                    assert r.holds[(t0 + 2 * i + 1) % 4] == t0 + 2 * i + 1
                yield from wait(barS, s0 + i)
                assert S[0] in (("S", e, i), ("P", e, i)) and (i == 0 or O[0] == (e, i))
                yield
                if barP.pending == 1:
                    S[0] = ("P", e, i)
                barP.arrive()
                yield
            t0, s0 = t0 + 2 * n, s0 + n
            if n:
                yield from wait(barO, done)
                assert O[0] == (e, n)
                done += 1
                yield
                assert O[0] == (e, n)
                barF.arrive()
    for a in (loads(), issues(), softmax(), softmax()):
        m.add(a)
    m.run()


def test_one_query_tile_over_items():
    for seed in range(250):
        rnd = random.Random(seed)
        few_model([rnd.choice([0, 1, 1, 2, 3, 6]) for _ in range(rnd.randint(1, 8))], seed)


def weigh_many_model(units, seed, slots=4, groups=4, buffers=4, sets=2):
    """k_weigh_many: units of that many query tiles, two issuers in turn; loads and products run on into
    the next unit, the groups meet at a unit's end.  `sets`: of sums, in turn."""
    m = Loose(seed)
    r = Ring(m, slots)
    barU, barK, barF = [Bar(1), Bar(1)], [Bar(1), Bar(1)], [Bar(2 * groups + 3), Bar(2 * groups + 3)]
    barS, barE = [Bar(1) for _ in range(buffers)], [Bar(2) for _ in range(buffers)]
    unit, K, S, sums_of = [None] * 2, [None] * 2, [None] * buffers, [[None] * groups for _ in range(sets)]
    everyone, phases = Bar(2 * groups), [0] * (2 * groups)

    def plans():
        for e, n in enumerate(units):
            if e >= 2:
                yield from wait(barF[e % 2], e // 2 - 1)
            unit[e % 2] = e
            barU[e % 2].arrive()
            K[e % 2] = None
            barK[e % 2].arrive(tx=1)

            def land(e=e):
                K[e % 2] = e
                barK[e % 2].complete(1)
            m.copy(land)
            yield
        for e in range(max(0, len(units) - 2), len(units)):
            yield from wait(barK[e % 2], e // 2)

    def loads():
        t = 0
        for e, n in enumerate(units):
            yield from wait(barU[e % 2], e // 2)
            assert unit[e % 2] == e, "another unit"
            barF[e % 2].arrive()
            for _ in range(n):
                yield from r.load(t)
                t += 1
        for u in range(max(0, t - slots), t):
            yield from r.landed(u)

    def issues(w):
        t = 0
        for e, n in enumerate(units):
            yield from wait(barU[e % 2], e // 2)
            assert unit[e % 2] == e, "another unit"
            yield from wait(barK[e % 2], e // 2)
            for _ in range(n):
                if t % 2 == w:
                    yield from r.landed(t)
                    if t >= buffers:
                        yield from wait(barE[t % buffers], t // buffers - 1)

                    def done(over=r.use(t), t=t, e=e):
                        assert K[e % 2] == e, "other keys"
                        over()
                        S[t % buffers] = t
                    m.mma(done, barS[t % buffers].arrive)
                    r.release(t)
                    yield
                t += 1
            m.mma(barF[e % 2].arrive)
        for u in range(max(0, t - slots), t):
            if u % 2 == w:
                yield from wait(r.empty[u % slots], u // slots)
        for e in range(max(0, len(units) - 2), len(units)):
            yield from wait(barF[e % 2], e // 2)

    def sums(x, me):
        def take(e):
            yield from wait(barU[e % 2], e // 2)
            assert unit[e % 2] == e, "another unit"
            yield
            barF[e % 2].arrive()
        t = 0
        yield from take(0)
        for e, n in enumerate(units):
            j = (x + groups - t % groups) % groups
            while j < n:
                u = t + j
                yield from wait(barS[u % buffers], u // buffers)
                assert S[u % buffers] == u, "scores of another tile"
                yield
                assert S[u % buffers] == u, "scores overwritten"
                barE[u % buffers].arrive()
                j += groups
            t += n
            if e + 1 < len(units):
                yield from take(e + 1)
            if me % 2 == 0 and x > 0:
                sums_of[e % sets][x] = e
            yield from meet(everyone, phases, me)
            if x == 0:
                for g in range(1, groups):
                    yield
                    assert sums_of[e % sets][g] == e, "sums of another unit"
    for a in [plans(), loads(), issues(0), issues(1)] + [sums(x, 2 * x + i) for x in range(groups) for i in range(2)]:
        m.add(a)
    m.run()


def test_weights_of_many_queries():
    for seed in range(150):
        rnd = random.Random(seed)
        weigh_many_model([rnd.choice([0, 1, 2, 3, 5, 9]) for _ in range(rnd.randint(1, 7))], seed)


def test_two_issuers_of_an_odd_ring_fail():
    """A slot's phases are then not one issuer's: it may ask for one that is two ahead."""
    assert fails(lambda seed: weigh_many_model([25], seed, slots=5), 400) > 0


def test_one_set_of_sums_fails():
    """A group that goes on writes its next sums while the last ones are read."""
    assert fails(lambda seed: weigh_many_model([1, 0, 2, 1, 1, 0, 1], seed, sets=1), 400) > 0


def weigh_few_model(run, seed):
    """k_weigh_few over (head, query tiles, whether the head ends) of each key tile of a run."""
    m = Loose(seed)
    r = Ring(m, 2)
    qfull, qempty = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
    barS, barE = [Bar(1) for _ in range(4)], [Bar(2) for _ in range(4)]
    Q, Qusers, S = [None, None], [0, 0], [None] * 4

    def loads():
        t, i, fresh = 0, 0, True
        for head, nq, last in run:
            for qt in range(nq):
                if nq > 1 or fresh:
                    if i >= 2:
                        yield from wait(qempty[i & 1], i // 2 - 1)
                    assert not Qusers[i & 1]
                    qfull[i & 1].arrive(tx=1)

                    def land(i=i, what=(head, qt)):
                        Q[i & 1] = what
                        qfull[i & 1].complete(1)
                    m.copy(land)
                    i += 1
                    yield
                if qt == 0:
                    yield from r.load(t)
            t += 1
            fresh = last
        for k in range(max(0, i - 2), i):
            yield from wait(qfull[k & 1], k // 2)
        for u in range(max(0, t - 2), t):
            yield from r.landed(u)

    def issues():
        t, i, u, fresh = 0, 0, 0, True
        for head, nq, last in run:
            for qt in range(nq):
                if nq > 1 or fresh:
                    yield from wait(qfull[i & 1], i // 2)
                    i += 1
                if qt == 0:
                    yield from r.landed(t)
                if u >= 4:
                    yield from wait(barE[u % 4], u // 4 - 1)
                b = (i - 1) & 1
                assert Q[b] == (head, qt), "other queries"
                Qusers[b] += 1

                def done(over=r.use(t), b=b, u=u):
                    over()
                    Qusers[b] -= 1
                    S[u % 4] = u
                m.mma(done, barS[u % 4].arrive)
                if nq > 1 or last:
                    m.mma(qempty[b].arrive)
                if qt + 1 == nq:
                    r.release(t)
                u += 1
                yield
            t += 1
            fresh = last
        for k in range(max(0, i - 2), i):
            yield from wait(qempty[k & 1], k // 2)
        yield from r.end(t)

    def sums():
        for u in range(sum(nq for _, nq, _ in run)):
            yield from wait(barS[u % 4], u // 4)
            assert S[u % 4] == u
            yield
            assert S[u % 4] == u
            barE[u % 4].arrive()
    for a in (loads(), issues(), sums(), sums()):
        m.add(a)
    m.run()


def test_weights_of_few_queries():
    for seed in range(200):
        rnd = random.Random(seed)
        run, n = [], rnd.randint(1, 5)
        for head in range(n):
            nq, k = rnd.choice([1, 1, 1, 2, 3]), rnd.randint(1, 5)
            run += [(head, nq, i + 1 == k) for i in range(k)]
        weigh_few_model(run, seed)
