"""The plan of a run that is refilled (CPU): how the warps of a kernel over pages meet around it, over
random interleavings, and which barriers the sources use for that.

A run of more items than are planned at a time is planned in batches: the warps that have read one meet,
one of them plans the next, they meet again.  Warps without a role go straight to the barrier at the kernel's
end, and must not be counted where the others meet."""
import glob
import os
import re

import pytest

from test_ops_protocol_model import Bar, wait
from test_paged_models import Loose, Ring, fails

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_rnn_gb300", "csrc")


def test_roles_meet_at_barriers_of_their_own():
    """Barrier 0 is the block's, which __syncthreads() names; a role that asks for it meets whoever is at one."""
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        assert not re.search(r"bar(rier)?\.(cta\.)?(sync|arrive|red[.a-z]*)\s+(0\b|[^;]*\"n\"\(0\))", text), path


class Block:
    """A block's barrier as the hardware counts it: complete when all that have not left are there."""

    def __init__(self, n):
        self.alive, self.here, self.phase = n, [], 0

    def meet(self, place):
        self.here.append(place)
        phase = self.phase
        while self.phase == phase:
            if len(self.here) >= self.alive:
                assert len(set(self.here)) == 1, "some of a meeting are somewhere else"
                self.here, self.phase = [], self.phase + 1
            else:
                yield

    def leave(self):
        self.alive -= 1


def refill_model(work, batch, seed, readers=2, idle=2, named=True, second=True):
    """A loading warp that plans, an issuing one, `readers` that take the results of n tiles of each item, and
    idle ones.  named: the roles have a barrier of their own; second: they meet again behind the plan."""
    m = Loose(seed)
    ring = Ring(m, 4)
    roles = 2 + readers
    end = Block(roles + idle)
    own = Block(roles) if named else end
    barS, barE = Bar(1), Bar(readers)
    plan = {"items": work[:batch], "more": len(work) > batch, "from": 0}

    def items(me, refill=None):
        """(index, tiles) of each item, read from the plan as the role goes."""
        while True:
            first, n = plan["from"], len(plan["items"])
            for i in range(n):
                assert plan["from"] == first and plan["items"] is not None, "the plan changed under its reader"
                yield first + i, plan["items"][i]
            assert plan["from"] == first, "the plan changed under its reader"
            if not plan["more"]:
                return
            yield from own.meet("read")
            if refill:
                refill(first + n)
                yield
            if second:
                yield from own.meet("planned")

    def refill(first):
        plan.update(items=None)
        plan.update({"from": first, "items": work[first:first + batch], "more": len(work) > first + batch})

    def ended(place="end"):
        yield from end.meet(place)
        end.leave()

    def loads():
        t = 0
        for step in items(0, refill):
            if step is None:
                yield
                continue
            for _ in range(step[1]):
                yield from ring.load(t)
                t += 1
        for u in range(max(0, t - 4), t):
            yield from ring.landed(u)
        yield from ended()

    def issues():
        t = 0
        for step in items(1):
            if step is None:
                yield
                continue
            for _ in range(step[1]):
                yield from ring.landed(t)
                if t:
                    yield from wait(barE, t - 1)
                m.mma(ring.use(t), barS.arrive)
                ring.release(t)
                t += 1
        yield from ring.end(t)
        yield from ended()

    done = [[] for _ in range(readers)]

    def reads(r):
        t = 0
        for step in items(2 + r):
            if step is None:
                yield
                continue
            for _ in range(step[1]):
                yield from wait(barS, t)
                yield
                barE.arrive()
                t += 1
            done[r].append(step)
        yield from ended()
    for actor in [loads(), issues()] + [reads(r) for r in range(readers)] + [ended() for _ in range(idle)]:
        m.add(actor)
    m.run()
    assert all(d == list(enumerate(work)) for d in done), "items left out or taken twice"


WORK = [[1], [1] * 5, [2, 0, 1, 3, 1, 1, 0], [0] * 9, [1, 2, 3, 4, 1, 0, 2, 1, 1, 1, 1]]


@pytest.mark.parametrize("batch", [1, 2, 4, 16])
@pytest.mark.parametrize("idle", [0, 2])
def test_plans_are_refilled(batch, idle):
    for work in WORK:
        for seed in range(12):
            refill_model(work, batch, seed, idle=idle)


def test_the_block_s_barrier_fails():
    """Warps that are at the kernel's end are taken for ones that have read the plan."""
    assert fails(lambda seed: refill_model([1] * 5, 2, seed, named=False)) > 0


def test_one_meeting_fails():
    """A warp that reads ahead of the new plan."""
    assert fails(lambda seed: refill_model([1] * 5, 2, seed, second=False)) > 0
