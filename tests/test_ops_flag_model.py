"""The flags that pass the decay backward's running sums from one head's CTA to the next, on the CPU.

The operations that a warp makes around a flag are read from the kernel's source and run in a
model of what the memory model promises: a lane knows of another CTA's writes through its own
acquire, or through a barrier with a lane that knows of them; a shuffle passes a value on and
orders nothing.
"""
import os
import random
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_rnn_gb300", "csrc",
                      "gdn_decay.cu")


def body(name):
    """The text between the braces of function `name`."""
    with open(SOURCE) as f:
        s = f.read()
    at = s.index("{", re.search(r"\b%s\(" % name, s).end())
    depth, i = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(s[i], 0)
        if depth == 0:
            return s[at:i + 1]
        i += 1


# ---- order ----------------------------------------------------------------------------------

def operations(text):
    """Acquires, barriers and shuffles in the order of the text."""
    return re.findall(r"ld\.acquire|__syncwarp|__shfl_sync", text)


def knowing_lanes(ops):
    """Lanes that know, behind `ops`, of what the flag's writer wrote before it (lane 0 alone acquires)."""
    knows = [False] * 32
    for op in ops:
        if op == "ld.acquire":
            knows[0] = True
        elif op == "__syncwarp":
            knows = [any(knows)] * 32
    return sum(knows)


def test_every_lane_may_read_behind_a_flag():
    ops = operations(body("wait_flag"))
    assert ops.count("ld.acquire") == 1
    assert knowing_lanes(ops) == 32


def test_a_shuffle_alone_orders_nothing():
    assert knowing_lanes(["ld.acquire", "__shfl_sync"]) == 1
    assert knowing_lanes(["__syncwarp", "ld.acquire"]) == 1


# ---- bounds ---------------------------------------------------------------------------------

def waits_on_flags_that_nobody_sets(call, wait, chunks):
    """How often a warp waits for its whole limit over a walk's chunks: the call passes on whether a wait has
    given up before, and the wait's loop asks for it first."""
    guarded = "w.ok" in re.search(r"wait_flag\((.*)\)", call).group(1) and re.search(r"\bif \([^;{]*\bok\b", wait)
    ok, waits = True, 0
    for _ in range(chunks):
        if ok or not guarded:
            waits += 1
            ok = False
    return waits


def test_a_walk_waits_for_one_limit_at_most():
    call = re.search(r"w\.ok = [^;]*wait_flag\([^;]*;", body("walk")).group(0)
    assert waits_on_flags_that_nobody_sets(call, body("wait_flag"), 512) == 1


def test_a_wait_that_does_not_ask_repeats_its_limit():
    assert waits_on_flags_that_nobody_sets("w.ok = wait_flag(flag, g) && w.ok;", "{ if (lane == 0) loop; }", 512) == 512


# ---- places -----------------------------------------------------------------------------------

def run_cta_order(order, places_by, sms, group, chunks=3):
    """CTAs start in `order`, one to an SM, and stay until they are done; the CTA at a place waits, chunk by chunk, for
    the place before it of its group.  places_by: "index" (a CTA's own) or "counter" (the next one when it starts).
    True if all of them end."""
    waiting, counter, running, done = list(order), 0, {}, {}
    while True:
        while waiting and len(running) < sms:
            cta = waiting.pop(0)
            place = cta if places_by == "index" else counter
            counter += 1
            running[place] = 0
        if not running:
            return not waiting
        before = dict(running)
        for place, c in before.items():
            ahead = done.get(place - 1, running.get(place - 1, 0))
            if place % group == 0 or ahead > c:
                running[place] = c + 1
        for place in [p for p, c in running.items() if c == chunks]:
            done[place] = running.pop(place)
        if running == before:
            return False


def places_of_the_kernel():
    text = body("decay_block")
    place = re.search(r"const int hd = (\w+(?:\.\w+)?) % a\.Hv", text).group(1)
    return "index" if place == "blockIdx.x" else "counter" if re.search(r"atomicAdd\(a\.ticket, 1\)", text) else None


def test_sums_pass_on_in_any_order_of_starts():
    rnd = random.Random(1)
    for _ in range(200):
        n, group = 24, rnd.choice([2, 3, 4, 8])
        order = rnd.sample(range(n), n)
        assert run_cta_order(order, places_of_the_kernel(), rnd.choice([1, 2, 5, 16]), group)


def test_places_by_index_need_starts_in_order():
    assert run_cta_order(range(24), "index", 2, 4)
    assert not run_cta_order(reversed(range(24)), "index", 2, 4)
