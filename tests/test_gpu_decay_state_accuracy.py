"""Returned states of decayed linear attention hold fp32 whatever the newer rows are.

A few rows of a sequence are not zero, all in different chunks, so a state is a sum of a few weighted
outer products and its error can be bounded tightly.  The decays are powers of two, so decay times
distance is exact.  Per term, relative to its size: expf 2 units in the last place (2 * 2^-23), the
row's scaling 2^-24, the three bf16 terms 2^-24, the products' sum 2 * 2^-24, a weight to the
state's end from a segment's one more expf and product (2 * 2^-23 + 2^-24).  Sums: 2^-23 of the terms' sizes for each
of at most 8 additions of parts that are not zero.  Together below 14 * 2^-23 of the sum of the terms' sizes,
1.7e-6.  Every further segment on the way multiplies by an expf (2 * 2^-23) and adds (2 * 2^-24): 3 * 2^-23 for each
of at most one segment to a chunk.  Terms below fp32's smallest normal number may be lost: 2^-126 for each of 8.
Two bf16 terms instead of three would be off by up to 2^-16, 1.5e-5.
"""
import pytest
import torch

import test_gpu_decay as D
from oracle import ops

pytestmark = pytest.mark.gpu

TOL = 14 * 2.0 ** -23


def sparse(T, rows, Hk, Hv, seed):
    gen = torch.Generator().manual_seed(seed)
    x = dict(q=torch.zeros(T, Hk, 128), k=torch.zeros(T, Hk, 128), v=torch.zeros(T, Hv, 128), dO=torch.zeros(T, Hv, 128))
    for n, t in x.items():
        t[rows] = torch.randn(len(rows), *t.shape[1:], generator=gen)
        x[n] = t.bfloat16()
    return x


def close(x, ref, size, what, segments):
    err = (x.double().cpu() - ref).abs()
    bad = ~(err <= (TOL + 3 * 2.0 ** -23 * (segments - 1)) * size + 8 * 2.0 ** -126)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst {float((err / size).nan_to_num().max()):.1e}"


# rows that are not zero, and how many tokens of zeros lie behind (forward) or before (backward) them
@pytest.mark.parametrize("T,rows", [(900, [3]), (900, [0, 130, 260]), (900, [100, 600, 899]), (2500, [7, 140]), (200, [5])])
@pytest.mark.parametrize("decays", [(-2.0 ** -6, -2.0 ** -7), (-2.0 ** -5, 0.0)])
def test_old_rows_alone(gdn_lib, T, rows, decays):
    Hk, Hv = 1, 2
    w = torch.tensor(decays)
    fwd, bwd = sparse(T, rows, Hk, Hv, T), sparse(T, [T - 1 - r for r in rows], Hk, Hv, T + 1)
    a = lambda t: t.abs()
    ref, size = (ops.decay_fwd(f(fwd["q"]), f(fwd["k"]), f(fwd["v"]), w, None, [T])[1] for f in (lambda t: t, a))
    gref, gsize = (ops.decay_bwd(f(bwd["q"]), f(bwd["k"]), f(bwd["v"]), w, None, f(bwd["dO"]), None, [T])[3]
                   for f in (lambda t: t, a))
    for most in (1, T):  # one segment, and as many as the call takes
        args = dict(cu_seqlens=D.cu([T]), max_seqlen=most)
        n = -(-most // 128)
        _, hT = gdn_lib.decay_fwd(fwd["q"].cuda(), fwd["k"].cuda(), fwd["v"].cuda(), w.cuda(), **args)
        close(hT, ref, size, f"hT, max_seqlen {most}", n)
        dh0 = gdn_lib.decay_bwd(bwd["q"].cuda(), bwd["k"].cuda(), bwd["v"].cuda(), w.cuda(), None, bwd["dO"].cuda(), **args)[3]
        close(dh0, gref, gsize, f"dh0, max_seqlen {most}", n)
