"""Gradients of rows that see few keys, where delta = dO . o from a rounded o would show.

Tolerance.  Two roundings to bf16 remain on the way to dq and dk, of ds and of the
result.  Each is off by at most half of 2^-7 of a value's power of two, in the root
mean square by at most 2^-8 / sqrt(3) of the value, so both by at most 2^-8 sqrt(2 / 3) =
3.2e-3 in the 2-norm of many values; a tenth is added for the sample.
"""
import pytest
import torch

import test_gpu_attn as A
from oracle import ops

pytestmark = pytest.mark.gpu

TOL = 1.1 * 2.0 ** -8 * (2.0 / 3.0) ** 0.5


@pytest.mark.parametrize("lens,Hq,Hk", [([2] * 20, 4, 2), ([3, 1, 0, 2] * 8, 6, 2), ([8, 5, 9, 7] * 4, 4, 4),
                                        ([2] * 40 + [4] * 30, 8, 1), ([30, 2, 17], 16, 4)])
def test_two_norm_of_gradients(gdn_lib, lens, Hq, Hk):
    x = A.make(lens, lens, Hq, Hk, seed=len(lens))
    d = {n: t.cuda() for n, t in x.items()}
    args = dict(cu_q=A.cu(lens), cu_k=A.cu(lens))
    o, lse = gdn_lib.attn_fwd(d["q"], d["k"], d["v"], **args)
    got = gdn_lib.attn_bwd(d["q"], d["k"], d["v"], o, lse, d["dO"], **args)
    r = ops.attn(x["q"], x["k"], x["v"], lens, A.cu(lens).tolist()[:-1], lens, 128 ** -0.5, x["dO"])
    for n, g in zip(("dq", "dk", "dv"), got):
        err = float((g.double().cpu() - r[n]).norm() / r[n].norm())
        assert err <= TOL, f"{n}: {err:.2e} > {TOL:.2e}"


def test_cached_keys_and_batched_layout(gdn_lib):
    """Rows that see one to eight keys and more beside rows that see none; no starts given."""
    ql, kl = [4, 12, 6], [6, 3, 20]
    A.check(gdn_lib, A.make(ql, kl, 4, 2, seed=5), ql, kl)
    B, T = 6, 5
    x = A.make([T] * B, [T] * B, 4, 2, seed=6)
    d = {n: t.cuda().view(B, T, -1, 128) for n, t in x.items()}
    o, lse = gdn_lib.attn_fwd(d["q"], d["k"], d["v"])
    got = gdn_lib.attn_bwd(d["q"], d["k"], d["v"], o, lse, d["dO"])
    r = ops.attn(x["q"], x["k"], x["v"], [T] * B, [T * b for b in range(B)], [T] * B, 128 ** -0.5, x["dO"],
                 A.eps_of(x, 128 ** -0.5))
    for n, g in zip(("dq", "dk", "dv"), got):
        A.close(g.flatten(0, 1), r[n], r[n + "_tol"], n)
