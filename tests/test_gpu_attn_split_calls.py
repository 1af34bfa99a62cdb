"""Attention calls whose keys are split over CTAs, in each of the two kernels that do it:
parts of prompts over long caches, with sequences of one query tile and of none among
them, and a few tokens each.  The bounds are those of the attention tests.
"""
import pytest
import torch

import test_gpu_attn as A
from oracle import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ql,used,cap,Hq,Hk", [
    ([300, 5, 0, 1], [6000, 4999, 700, 1], 6000, 4, 2),       # several query tiles beside one
    ([260, 64], [257, 5000], 5000, 6, 2),                     # groups of three; more queries than keys
    ([700], [4100], 4100, 2, 2),
    ([7, 0, 3, 64], [5000, 0, 130, 64], 5000, 4, 2),          # one tile each
    ([16] * 5, [4000, 3999, 16, 17, 129], 4000, 8, 1),        # whole tiles of 16 tokens
    ([1] * 6, [9000, 1, 128, 129, 0, 640], 9000, 128, 1),     # a tile is one token
])
def test_keys_split(gdn_lib, ql, used, cap, Hq, Hk):
    n = len(ql)
    assert gdn_lib.attn_workspace_bytes(0, n, sum(ql), n * cap, cap, Hq, Hk) > 256  # parts to join
    x = A.make(ql, [cap] * n, Hq, Hk, seed=sum(ql))
    for name in ("k", "v"):  # what lies past the used rows is never seen
        c = x[name].view(n, cap, Hk, 128)
        for b, m in enumerate(used):
            c[b, m:] = float("nan")
    clean = {k: torch.nan_to_num(t) for k, t in x.items()}
    r = ops.attn(x["q"], clean["k"], clean["v"], ql, [b * cap for b in range(n)], used, 128 ** -0.5,
                 eps=A.eps_of(clean, 128 ** -0.5))
    args = dict(cu_q=A.cu(ql), cu_k=A.cu([cap] * n), k_len=torch.tensor(used, dtype=torch.int32).cuda())
    q, k, v = x["q"].cuda(), x["k"].cuda(), x["v"].cuda()
    runs = [gdn_lib.attn_fwd(q, k, v, max_k=cap, **args) for _ in range(2)]
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    A.close(runs[0][0], r["o"], r["o_tol"], "o")
    A.close(runs[0][1], r["lse"], r["lse_tol"], "lse")
    o, lse = gdn_lib.attn_fwd(q, k, v, max_k=1, **args)  # (max_k only steers the work)
    A.close(o, r["o"], r["o_tol"], "o")
    A.close(lse, r["lse"], r["lse_tol"], "lse")


@pytest.mark.parametrize("lens,Hq,Hk", [([640, 1, 0, 333], 4, 2), ([100] * 9, 6, 2), ([5, 128, 129, 600], 2, 2)])
def test_short_prompts(gdn_lib, lens, Hq, Hk):
    """Prompts of at most five key tiles, several query tiles to a sequence."""
    A.check(gdn_lib, A.make(lens, lens, Hq, Hk, seed=sum(lens)), lens, lens)
