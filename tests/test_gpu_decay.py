"""Linear attention with a decay for each head against its 64-bit recurrence and adjoint.

Tolerances, element by element.  Let A be the same operation on the inputs'
absolute values (every sum's sum of sizes).  The masked scores and the entering
state of a chunk are rounded to bf16 (unit roundoff 2^-8 of each term, so 2^-8 A
in all) and the result to bf16 (2^-8 |o|); fp32 sums add at most 2^-23 per
addition.  The states and their gradients keep two bf16 terms of each scaled row
(2^-16) and fp32 sums over the sequence's tokens.
"""
import pytest
import torch

from oracle import ops

pytestmark = pytest.mark.gpu


def make(lens, Hk, Hv, seed, h0=True, fast=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    n, total = len(lens), sum(lens)
    bf = lambda x: x.bfloat16()
    return dict(q=bf(r(total, Hk, 128) * 0.3), k=bf(r(total, Hk, 128) * 0.3), v=bf(r(total, Hv, 128)),
                decay=-torch.rand(Hv, generator=gen) * (30.0 if fast else 0.1),
                h0=r(n, Hv, 128, 128) if h0 else None, dO=bf(r(total, Hv, 128)), dhT=r(n, Hv, 128, 128))


def cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def close(x, ref, size, what, rounded, longest):
    x, ref, size = x.detach().cpu().double(), ref, size
    sums = (longest + 256) * 2.0 ** -23
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + sums) * size if rounded else (2.0 ** -16 + sums) * size
    bad = ((x - ref).abs() > 1.02 * tol + 1e-30) | ~torch.isfinite(x)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound"


def check_fwd(gdn, x, lens, o, hT):
    a = lambda t: None if t is None else t.abs()
    ro, rh = ops.decay_fwd(x["q"], x["k"], x["v"], x["decay"], x["h0"], lens)
    ao, ah = ops.decay_fwd(a(x["q"]), a(x["k"]), a(x["v"]), x["decay"], a(x["h0"]), lens)
    m = max(lens)
    close(o, ro, ao, "o", True, m)
    close(hT, rh, ah, "hT", False, m)


def check_bwd(gdn, x, lens, got):
    a = lambda t: None if t is None else t.abs()
    names = ("q", "k", "v")
    ref = ops.decay_bwd(*[x[n] for n in names], x["decay"], x["h0"], x["dO"], x["dhT"], lens)
    size = ops.decay_bwd(*[a(x[n]) for n in names], x["decay"], a(x["h0"]), a(x["dO"]), a(x["dhT"]), lens)
    for n, g, r, s in zip(("dq", "dk", "dv", "dh0"), got, ref, size):
        close(g, r, s, n, n != "dh0", max(lens))


CASES = [([1], 1, 1), ([127], 1, 2), ([128], 2, 2), ([129], 1, 1), ([300, 1, 65, 0], 2, 2), ([0, 513, 0], 1, 3),
         ([700], 1, 1), ([64, 128, 200, 1, 1, 1], 1, 4)]


@pytest.mark.parametrize("lens,Hk,Hv", CASES)
@pytest.mark.parametrize("h0", [True, False])
def test_packed_sequences(gdn_lib, lens, Hk, Hv, h0):
    x = make(lens, Hk, Hv, seed=sum(lens) + Hv, h0=h0)
    d = {k: None if t is None else t.cuda() for k, t in x.items()}
    args = dict(cu_seqlens=cu(lens), max_seqlen=max(lens))
    o, hT = gdn_lib.decay_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], **args)
    got = gdn_lib.decay_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["dO"], d["dhT"], **args)
    check_fwd(gdn_lib, x, lens, o, hT)
    check_bwd(gdn_lib, x, lens, got)


@pytest.mark.parametrize("lens", [[900, 300], [40, 1100, 129]])
def test_one_segment_and_several_agree(gdn_lib, lens):
    """max_seqlen only steers the split: with 1 the longest sequence is one segment."""
    x = make(lens, 1, 2, seed=5)
    d = {k: t.cuda() for k, t in x.items()}
    for most in (1, max(lens)):
        args = dict(cu_seqlens=cu(lens), max_seqlen=most)
        o, hT = gdn_lib.decay_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], **args)
        got = gdn_lib.decay_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["dO"], d["dhT"], **args)
        check_fwd(gdn_lib, x, lens, o, hT)
        check_bwd(gdn_lib, x, lens, got)


def test_fast_and_zero_decays(gdn_lib):
    lens = [260, 500]
    x = make(lens, 1, 4, seed=6, fast=True)
    x["decay"][0] = 0.0      # a plain sum
    x["decay"][1] = -200.0   # nothing is kept
    d = {k: t.cuda() for k, t in x.items()}
    args = dict(cu_seqlens=cu(lens), max_seqlen=500)
    o, hT = gdn_lib.decay_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], **args)
    check_fwd(gdn_lib, x, lens, o, hT)
    check_bwd(gdn_lib, x, lens,
              gdn_lib.decay_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["dO"], d["dhT"], **args))


def test_batched_layout_and_parts_of_one_buffer(gdn_lib):
    B, T, Hk, Hv = 2, 150, 2, 4
    x = make([T] * B, Hk, Hv, seed=7)
    qkv = torch.cat([x["q"].flatten(1), x["k"].flatten(1), x["v"].flatten(1)], 1).cuda().view(B, T, -1)
    q, k, v = qkv.split([Hk * 128, Hk * 128, Hv * 128], 2)
    q, k, v = q.view(B, T, Hk, 128), k.view(B, T, Hk, 128), v.view(B, T, Hv, 128)
    w, h0 = x["decay"].cuda(), x["h0"].cuda()
    o, hT = gdn_lib.decay_fwd(q, k, v, w, h0)
    assert o.shape == (B, T, Hv, 128)
    check_fwd(gdn_lib, x, [T] * B, o.flatten(0, 1), hT)
    got = gdn_lib.decay_bwd(q, k, v, w, h0, x["dO"].cuda().view(B, T, Hv, 128), x["dhT"].cuda())
    check_bwd(gdn_lib, x, [T] * B, [got[0].flatten(0, 1), got[1].flatten(0, 1), got[2].flatten(0, 1), got[3]])


def test_neighbouring_rows_do_not_matter(gdn_lib):
    """A sequence beside one of NaN and infinities (its last chunk's tile runs into it)."""
    lens = [130, 90, 200]
    x = make(lens, 1, 2, seed=8)
    bad = slice(130, 220)
    d = {k: t.clone().cuda() for k, t in x.items()}
    for n in ("q", "k", "v", "dO"):
        d[n][bad] = float("nan")
        d[n][135:140] = float("inf")
    keep = torch.tensor([i for i in range(sum(lens)) if not 130 <= i < 220])
    y = {n: (t[keep] if n in ("q", "k", "v", "dO") else t[[0, 2]] if n in ("h0", "dhT") else t) for n, t in x.items()}
    for most in (1, 200):
        args = dict(cu_seqlens=cu(lens), max_seqlen=most)
        o, hT = gdn_lib.decay_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], **args)
        check_fwd(gdn_lib, y, [130, 200], o.cpu()[keep], hT[[0, 2]])
        got = gdn_lib.decay_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["dO"], d["dhT"], **args)
        check_bwd(gdn_lib, y, [130, 200], [g.cpu()[keep] for g in got[:3]] + [got[3][[0, 2]]])


def test_no_rows_pass_the_state_on(gdn_lib):
    x = make([0, 0], 1, 2, seed=9)
    d = {k: t.cuda() for k, t in x.items()}
    o, hT = gdn_lib.decay_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], cu_seqlens=cu([0, 0]), max_seqlen=0)
    assert o.shape[0] == 0 and torch.equal(hT, d["h0"])
    got = gdn_lib.decay_bwd(d["q"], d["k"], d["v"], d["decay"], None, d["dO"], d["dhT"], cu_seqlens=cu([0, 0]),
                            max_seqlen=0)
    assert torch.equal(got[3], d["dhT"])


def test_repeated_calls_are_equal(gdn_lib):
    lens = [700, 129]
    x = {k: t.cuda() for k, t in make(lens, 2, 4, seed=10).items()}
    args = dict(cu_seqlens=cu(lens), max_seqlen=700)
    runs = [gdn_lib.decay_bwd(x["q"], x["k"], x["v"], x["decay"], x["h0"], x["dO"], x["dhT"], **args)
            for _ in range(2)]
    assert all(torch.equal(a, b) for a, b in zip(*runs))
