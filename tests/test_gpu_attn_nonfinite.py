"""Scores that are not numbers, or too large for fp32: the rows that see them are NaN, output and
log-sum, as a softmax in fp32 has it, however the keys are split; every other row keeps its value.

NaN is exact, so it needs no tolerance; the other rows have the bounds of the attention tests.
"""
import pytest
import torch

import test_gpu_attn as A
from oracle import ops

pytestmark = pytest.mark.gpu

# queries, used keys, capacity, heads, max_k (1: a single split in the kernel that takes the call)
CASES = [
    ([1, 1, 1], [9000, 300, 9000], 9000, 4, 2, 9000),     # single tokens, keys split
    ([1, 1, 1], [9000, 300, 9000], 9000, 4, 2, 1),        # not split
    ([300, 5], [6000, 4999], 6000, 4, 2, 6000),           # part of a prompt, keys split
    ([700, 300], [1500, 1200], 1500, 4, 2, 1),            # several query tiles, not split
    ([400, 130], [400, 130], 400, 4, 1, 400),             # short prompts
]


def run(gdn, x, ql, used, cap, most):
    n = len(ql)
    o, lse = gdn.attn_fwd(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), cu_q=A.cu(ql), cu_k=A.cu([cap] * n), max_k=most,
                          k_len=torch.tensor(used, dtype=torch.int32).cuda())
    return o.cpu(), lse.cpu()


def check(gdn, x, clean, hit, ql, used, cap, most):
    """hit [rows, heads]: rows whose scores are not numbers."""
    o, lse = run(gdn, x, ql, used, cap, most)
    r = ops.attn(clean["q"], clean["k"], clean["v"], ql, [b * cap for b in range(len(ql))], used, 128 ** -0.5,
                 eps=A.eps_of(clean, 128 ** -0.5))
    assert bool(torch.isnan(o[hit]).all()), f"o: {int((~torch.isnan(o[hit])).sum())} finite values of {o[hit].numel()}"
    assert bool(torch.isnan(lse[hit]).all()), f"lse: {lse[hit][~torch.isnan(lse[hit])][:4].tolist()}"
    A.close(o[~hit], r["o"][~hit], r["o_tol"][~hit], "o of the other rows")
    A.close(lse[~hit], r["lse"][~hit], r["lse_tol"][~hit], "lse of the other rows")


def seeing(ql, used, Hq, Hk, seq, head, key):
    """Rows of sequence `seq` that see `key` of key head `head`."""
    hit = torch.zeros(sum(ql), Hq, dtype=torch.bool)
    G, q0 = Hq // Hk, sum(ql[:seq])
    for i in range(ql[seq]):
        if key <= i + used[seq] - ql[seq]:
            hit[q0 + i, head * G:(head + 1) * G] = True
    return hit


@pytest.mark.parametrize("ql,used,cap,Hq,Hk,most", CASES)
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_a_cached_key(gdn_lib, ql, used, cap, Hq, Hk, most, where):
    x = A.make(ql, [cap] * len(ql), Hq, Hk, seed=31)
    key = {"first": 0, "middle": used[0] // 2, "last": used[0] - 1}[where]
    clean = {n: t.clone() for n, t in x.items()}
    x["k"][key, Hk - 1, 17] = float("nan")
    hit = seeing(ql, used, Hq, Hk, 0, Hk - 1, key)
    assert bool(hit.any())
    check(gdn_lib, x, clean, hit, ql, used, cap, most)


@pytest.mark.parametrize("ql,used,cap,Hq,Hk,most", CASES)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query(gdn_lib, ql, used, cap, Hq, Hk, most, value):
    """An infinity gives scores of both signs, of which the positive ones overflow."""
    x = A.make(ql, [cap] * len(ql), Hq, Hk, seed=32)
    clean = {n: t.clone() for n, t in x.items()}
    x["q"][ql[0] - 1, 1, 5] = value
    hit = torch.zeros(sum(ql), Hq, dtype=torch.bool)
    hit[ql[0] - 1, 1] = True
    check(gdn_lib, x, clean, hit, ql, used, cap, most)


@pytest.mark.parametrize("ql,used,cap,Hq,Hk,most", CASES)
def test_an_overflowed_score(gdn_lib, ql, used, cap, Hq, Hk, most):
    """One key's product with one row is 1e40, past fp32, with the others it is small."""
    x = A.make(ql, [cap] * len(ql), Hq, Hk, seed=33)
    row, key = ql[0] - 1, used[0] // 2
    x["q"][:, :, 3] = 0.0
    clean = {n: t.clone() for n, t in x.items()}
    x["q"][row, 0, 3] = 1e20
    x["k"][key, 0, 3] = 1e20
    # (the row's other scores: what the key's values in that place give them, made zero)
    x["k"][:key, 0, 3] = 0.0
    x["k"][key + 1:, 0, 3] = 0.0
    hit = torch.zeros(sum(ql), Hq, dtype=torch.bool)
    hit[row, 0] = True
    check(gdn_lib, x, clean, hit, ql, used, cap, most)


def test_every_visible_key(gdn_lib):
    """No number among a row's scores at all, in every split."""
    ql, used, cap, Hq, Hk = [1, 2], [8000, 700], 8000, 4, 2
    x = A.make(ql, [cap] * 2, Hq, Hk, seed=34)
    clean = {n: t.clone() for n, t in x.items()}
    x["k"][:used[0], 0] = float("nan")
    hit = seeing(ql, used, Hq, Hk, 0, 0, 0)
    for most in (cap, 1):
        check(gdn_lib, x, clean, hit, ql, used, cap, most)


def test_scores_of_minus_infinity(gdn_lib):
    """Keys that a row weighs with nothing: minus infinity is a score like any other."""
    ql, used, cap, Hq, Hk = [1, 1], [7000, 130], 7000, 2, 1
    x = A.make(ql, [cap] * 2, Hq, Hk, seed=35)
    x["q"][:, :, 9] = 1.0
    x["k"][:5000, 0, 9] = -float("inf")
    x["v"][:5000] = 0.0
    short = {"q": x["q"], "k": torch.cat([x["k"][5000:7000], x["k"][7000:7130]]),
             "v": torch.cat([x["v"][5000:7000], x["v"][7000:7130]])}
    r = ops.attn(short["q"], short["k"], short["v"], ql, [0, 2000], [2000, 130], 128 ** -0.5, eps=A.eps_of(short, 128 ** -0.5))
    for most in (cap, 1):
        o, lse = run(gdn_lib, x, ql, used, cap, most)
        A.close(o, r["o"], r["o_tol"], "o")
        A.close(lse, r["lse"], r["lse_tol"], "lse")
