"""Shuffles of a whole warp in the head norms' kernel are reached by the whole warp (CPU).

CUDA leaves a shuffle undefined (its values, and whether it ends) where a lane that its mask
names does not take part.  A step has four heads side by side in a warp, and with pages some of
them may be keys and the others values.  The conditions around each call of head_sum, whose
mask is the warp, are read from the source and evaluated lane by lane: all lanes have to
decide the same."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_rnn_gb300", "csrc")
SIDE, LANES = 4, 8


def conditions(source, call):
    """For each place of `call`, the conditions of the branches around it in its function, outermost first."""
    text = re.sub(r"//[^\n]*", "", source)
    found, open_ = [], []
    for m in re.finditer(r"[{}]|" + re.escape(call), text):
        if m.group() == "{":
            head = text[max(text.rfind(c, 0, m.start()) for c in ";{}") + 1:m.start()].strip()
            if head == "else" or head.startswith("else if"):
                head = "else of " + closed
            open_.append(head)
        elif m.group() == "}":
            closed = open_.pop()
        else:
            found.append(list(open_))
    return found


def truth(head, lane):
    """The value of an `if` in one lane."""
    inverse = head.startswith("else of ")
    cond = re.fullmatch(r"(?:else of )?if(?: constexpr)? \((.*)\)", head, re.S).group(1)
    cond = re.sub(r"!(?!=)", " not ", cond.replace("&&", " and ").replace("||", " or "))
    return bool(eval(cond, {}, lane)) != inverse


def lanes(Hq, Hk, paged, back, i):
    Hqk = Hq + Hk
    H = Hqk + Hk if paged else Hqk
    for lane in range(32):
        h = SIDE * i + lane // LANES
        yield dict(PAGED=paged, BACK=back, SIDE=SIDE, h=h, i=i, own=h < H, is_k=h >= Hq, Hqk=Hqk, H=H, normed=True,
                   lane=lane, l=lane % LANES, side=lane // LANES)


def branches():
    with open(os.path.join(CSRC, "gdn_rope.cu")) as f:
        source = f.read()
    start = source.index("k_rope(const __grid_constant__ RopeArgs a)")
    found = conditions(source[start:source.index("k_rope_dw", start)], "head_sum(")
    assert len(found) >= 3
    return [[h for h in place if h.startswith(("if", "else"))] for place in found]


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 1), (4, 1), (8, 1), (4, 2), (8, 2), (16, 2), (6, 3), (3, 1), (16, 4), (5, 5)])
@pytest.mark.parametrize("paged,back", [(False, False), (True, False), (False, True)])
def test_shuffles_have_their_whole_warp(Hq, Hk, paged, back):
    H = Hq + Hk * (2 if paged else 1)
    for place in branches():
        for i in range(-(-H // SIDE)):
            def reached(lane):
                return all(truth(head, lane) for head in place)
            takes = [reached(lane) for lane in lanes(Hq, Hk, paged, back, i)]
            assert len(set(takes)) == 1, f"step {i}: {sum(takes)} of 32 lanes reach a shuffle of them all: {place}"


def test_a_branch_on_the_head_fails():
    """Heads 2 (a key) and 3 (a value) are in one warp."""
    place = ["if (!BACK)", "if (!PAGED || h < Hqk)", "if (normed)"]
    takes = [all(truth(head, lane) for head in place) for lane in lanes(2, 1, True, False, 0)]
    assert 0 < sum(takes) < 32
