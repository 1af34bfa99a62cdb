"""A model of the split attention kernel's handshakes over random interleavings (CPU), on
the machine of the other kernels' models: one accumulator for the scores, whose product
is issued behind the P V that reads its place, P handed over by one barrier.
"""
import pytest

from test_ops_protocol_model import Bar, Machine, Ring, wait


def split_model(n, seed, early=False):
    """`early`: the next scores issued before P V of the tile that lies in their place."""
    m = Machine(seed)
    r = Ring(m, 4, 2 * n)
    barS, barP, barO = Bar(1), Bar(2), Bar(1)
    S, O = [None], [0]

    def issue():
        def scores(i):
            yield from r.arrived(2 * i)
            m.mma(r.use(2 * i), lambda: S.__setitem__(0, i), barS.arrive)
            r.release(2 * i)
        yield from scores(0)
        for i in range(n):
            if early and i + 1 < n:
                yield from scores(i + 1)
            yield from r.arrived(2 * i + 1)
            yield from wait(barP, i)

            def product(i=i):
                assert S[0] == i, "P overwritten before its product"
                O[0] = i + 1
            m.mma(r.use(2 * i + 1), product)
            r.release(2 * i + 1)
            if not early and i + 1 < n:
                yield from scores(i + 1)
            yield
        m.mma(barO.arrive)

    def compute():
        for i in range(n):
            yield from r.arrived(2 * i + 1)          # (a ragged V tile's rows are cleared)
            yield from wait(barS, i)
            assert S[0] == i and O[0] == i, "O rescaled beside its product"
            yield
            barP.arrive()
            yield
        yield from wait(barO, 0)

    for a in (r.producer(), issue(), compute(), compute()):
        m.add(a)
    m.run()


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 9])
def test_handshakes_hold(n):
    for seed in range(80):
        split_model(n, seed)


def test_scores_ahead_of_the_product_fail():
    failed = 0
    for seed in range(60):
        try:
            split_model(5, seed, early=True)
        except AssertionError:
            failed += 1
    assert failed > 0
