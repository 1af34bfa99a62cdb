"""Packed calls at the ends of their range: many sequences, sequences cut into
segments under shared heads, heads that keep nothing, rows past 32-bit offsets.

The bounds are those of the operators' own tests: tolerances derived there, element
by element, applied here to more shapes.
"""
import pytest
import torch

import test_gpu_attn as A
import test_gpu_decay as D
import test_gpu_step as S
from conftest import assert_rel
from oracle import ops

pytestmark = pytest.mark.gpu


def lengths(n, most, seed, empty=4):
    gen = torch.Generator().manual_seed(seed)
    lens = torch.randint(1, most + 1, (n,), generator=gen).tolist()
    for i in range(0, n, empty):
        lens[i] = 0
    return lens


# ---- many sequences: places are found beyond the first 32 -----------------------------

@pytest.mark.parametrize("n,most,Hq,Hk", [(33, 200, 4, 2), (75, 90, 6, 2), (130, 30, 1, 1)])
@pytest.mark.parametrize("cached", [False, True])
def test_attention_many_sequences(gdn_lib, n, most, Hq, Hk, cached):
    ql = lengths(n, most, seed=n)
    kl = [a + b for a, b in zip(ql, lengths(n, 300, seed=n + 1, empty=3))] if cached else ql
    A.check(gdn_lib, A.make(ql, kl, Hq, Hk, seed=n), ql, kl)


def test_attention_tokens_of_many_users(gdn_lib):
    """Split keys (two key heads and long caches) over more than 32 sequences."""
    rows, cap, Hq, Hk = 40, 6000, 4, 1
    gen = torch.Generator().manual_seed(21)
    used = torch.randint(0, 700, (rows,), generator=gen).tolist()
    used[0], used[35], used[39] = 0, cap, cap - 1
    x = A.make([1] * rows, [cap] * rows, Hq, Hk, seed=21)
    r = ops.attn(x["q"], x["k"], x["v"], [1] * rows, [b * cap for b in range(rows)], used, 128 ** -0.5,
                 eps=A.eps_of(x, 128 ** -0.5))
    q, k, v = x["q"].cuda(), x["k"].cuda(), x["v"].cuda()
    for most in (cap, 1):
        o, lse = gdn_lib.attn_fwd(q, k, v, cu_q=A.cu([1] * rows), cu_k=A.cu([cap] * rows), max_k=most,
                                  k_len=torch.tensor(used, dtype=torch.int32).cuda())
        A.close(o, r["o"], r["o_tol"], "o")
        A.close(lse, r["lse"], r["lse_tol"], "lse")


def decay_both(gdn, x, lens, most=None):
    d = {k: None if t is None else t.cuda() for k, t in x.items()}
    args = dict(cu_seqlens=D.cu(lens), max_seqlen=max(lens) if most is None else most)
    o, hT = gdn.decay_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], **args)
    got = gdn.decay_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["dO"], d["dhT"], **args)
    D.check_fwd(gdn, x, lens, o, hT)
    D.check_bwd(gdn, x, lens, got)


@pytest.mark.parametrize("n,most,Hk,Hv", [(33, 140, 1, 2), (70, 60, 1, 3), (32, 150, 2, 2)])
def test_decay_many_sequences(gdn_lib, n, most, Hk, Hv):
    decay_both(gdn_lib, D.make(lengths(n, most, seed=n), Hk, Hv, seed=n), lengths(n, most, seed=n))


def segments(gdn, backward, lens, Hk, Hv, most):
    """Whether the call cuts its sequences: only then does the workspace hold states."""
    whole = gdn.decay_workspace_bytes(backward, len(lens), sum(lens), 1, Hk, Hv)
    return gdn.decay_workspace_bytes(backward, len(lens), sum(lens), most, Hk, Hv) > whole


def test_decay_many_sequences_in_segments(gdn_lib):
    lens = [3] * 20 + [2000] + [0, 1] * 8 + [1500, 7]
    assert len(lens) > 32 and segments(gdn_lib, False, lens, 1, 1, 2000)
    decay_both(gdn_lib, D.make(lens, 1, 1, seed=22), lens, 2000)


# ---- shared heads over segments ---------------------------------------------------------

@pytest.mark.parametrize("Hk,Hv", [(1, 2), (1, 3), (2, 8)])
@pytest.mark.parametrize("lens", [[2100], [2600, 0, 900, 130]])
def test_decay_shared_heads_in_segments(gdn_lib, Hk, Hv, lens):
    assert segments(gdn_lib, True, lens, Hk, Hv, max(lens))
    decay_both(gdn_lib, D.make(lens, Hk, Hv, seed=Hv), lens)


# ---- a head that keeps nothing -----------------------------------------------------------

@pytest.mark.parametrize("lens", [[300, 1, 0, 140], [1700]])
def test_decay_of_minus_infinity(gdn_lib, lens):
    """exp(decay) is zero for both, so the results are the same ones."""
    x = {k: t.cuda() for k, t in D.make(lens, 1, 2, seed=23).items()}
    args = dict(cu_seqlens=D.cu(lens), max_seqlen=max(lens))
    runs = []
    for w in (-float("inf"), -1000.0):
        w = torch.tensor([w, -0.02]).cuda()
        state = x["h0"][:1].clone()
        runs.append([*gdn_lib.decay_fwd(x["q"], x["k"], x["v"], w, x["h0"], **args),
                     *gdn_lib.decay_bwd(x["q"], x["k"], x["v"], w, x["h0"], x["dO"], x["dhT"], **args),
                     gdn_lib.decay_step(x["q"][:1], x["k"][:1], x["v"][:1], w, state), state])
    for a, b in zip(*runs):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b)


# ---- rows past 32-bit offsets --------------------------------------------------------------

def test_decay_far_rows(gdn_lib):
    """A short sequence behind one of more than 2^31 values; the long one's first rows."""
    Hv, head, lens = 16, 200, [1_049_000, 300]
    total, last = sum(lens), slice(lens[0], None)
    assert lens[0] * Hv * 128 > 2 ** 31
    x = D.make([head, 300], 1, Hv, seed=24)
    x["dhT"][0] = 0.0
    d = {}
    for n in ("q", "k", "v", "dO"):
        d[n] = torch.zeros(total, *x[n].shape[1:], dtype=torch.bfloat16, device="cuda")
        d[n][:head], d[n][last] = x[n][:head].cuda(), x[n][head:].cuda()
    w, h0, dhT = x["decay"].cuda(), x["h0"].cuda(), x["dhT"].cuda()
    args = dict(cu_seqlens=D.cu(lens), max_seqlen=lens[0])
    cut = lambda t: torch.cat([t[:head], t[last]]).cpu()
    o, hT = gdn_lib.decay_fwd(d["q"], d["k"], d["v"], w, h0, **args)
    got = gdn_lib.decay_bwd(d["q"], d["k"], d["v"], w, h0, d["dO"], dhT, **args)
    hT[0] = ops.decay_fwd(x["q"], x["k"], x["v"], x["decay"], x["h0"], [head, 300])[1][0].float().cuda()  # (decayed on)
    D.check_fwd(gdn_lib, x, [head, 300], cut(o), hT)
    D.check_bwd(gdn_lib, x, [head, 300], [cut(g) for g in got[:3]] + [got[3]])


def test_attention_far_rows(gdn_lib):
    n, T, H = 1000, 1050, 16
    assert n * T * H * 128 > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(25)
    x = {k: torch.randn(n, T, H, 128, generator=gen, device="cuda", dtype=torch.bfloat16) for k in ("q", "k", "v", "dO")}
    o, lse = gdn_lib.attn_fwd(x["q"], x["k"], x["v"])
    got = gdn_lib.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"])
    for s in (0, 999):
        y = {k: t[s].cpu() for k, t in x.items()}
        r = ops.attn(y["q"], y["k"], y["v"], [T], [0], [T], 128 ** -0.5, y["dO"], A.eps_of(y, 128 ** -0.5))
        A.close(o[s], r["o"], r["o_tol"], "o")
        A.close(lse[s], r["lse"], r["lse_tol"], "lse")
        for k, g in zip(("dq", "dk", "dv"), got):
            A.close(g[s], r[k], r[k + "_tol"], k)


def test_attention_far_cache(gdn_lib):
    rows, cap, H = 3, 600_000, 16
    assert (rows - 1) * cap * H * 128 > 2 ** 31
    used = [5, 0, 1500]
    x = A.make([1] * rows, [sum(used)], H, H, seed=26)
    k = torch.full((rows, cap, H, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, float("nan"))
    at = 0
    for b, m in enumerate(used):
        k[b, :m], v[b, :m] = x["k"][at:at + m].cuda(), x["v"][at:at + m].cuda()
        at += m
    o, lse = gdn_lib.attn_fwd(x["q"].cuda().view(rows, 1, H, 128), k, v, k_len=torch.tensor(used, dtype=torch.int32).cuda())
    r = ops.attn(x["q"], x["k"], x["v"], [1] * rows, [0, 5, 5], used, 128 ** -0.5, eps=A.eps_of(x, 128 ** -0.5))
    A.close(o.flatten(0, 1), r["o"], r["o_tol"], "o")
    A.close(lse.flatten(0, 1), r["lse"], r["lse_tol"], "lse")


@pytest.mark.parametrize("delta", [True, False])
def test_step_far_slots(gdn_lib, delta):
    slots, n, Hv = [4199, 0, 2100], 4200, 32
    assert n * Hv * 128 * 128 > 2 ** 31
    x = S._rows(3, 16, Hv, 3, seed=27)
    state = torch.zeros(n, Hv, 128, 128, device="cuda")
    state[slots] = x["state"].cuda()
    d = {k: t.cuda() for k, t in x.items()}
    idx = torch.tensor(slots, dtype=torch.int32).cuda()
    if delta:
        o = gdn_lib.delta_step(d["q"], d["k"], d["v"], d["g"], d["beta"], state, idx)
        ro, rs = ops.delta_step(x["q"], x["k"], x["v"], x["g"], x["beta"], x["state"], [0, 1, 2])
    else:
        o = gdn_lib.decay_step(d["q"], d["k"], d["v"], d["decay"], state, idx)
        ro, rs = ops.decay_step(x["q"], x["k"], x["v"], x["decay"], x["state"], [0, 1, 2])
    assert_rel(o.float().cpu(), ro, S.O_TOL, "o")
    assert_rel(state[slots].cpu(), rs, S.S_TOL, "state")
