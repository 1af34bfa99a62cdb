"""Norms of query and key heads with the rotation, its gradients and the form that fills a cache's
pages, against their 64-bit definitions within bounds derived from the roundings (oracle.ops.rope)."""
import pytest
import torch

from oracle import ops

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(n, Hq, Hk, pairs, seed, norm=True, axes=1, far=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    x = dict(q=(1.5 * r(n, Hq, 128)).bfloat16(), k=(1.5 * r(n, Hk, 128)).bfloat16(), v=r(n, Hk, 128).bfloat16(),
             gq=r(n, Hq, 128).bfloat16(), gk=r(n, Hk, 128).bfloat16(),
             pos=torch.randint(-5, 4000, (axes, n) if axes > 1 else (n,), generator=gen).int() + far,
             freq=torch.exp2(-torch.arange(pairs, dtype=torch.float64) * 20 / max(pairs, 1)).float(),
             wq=1 + 0.2 * r(128) if norm else None, wk=1 + 0.2 * r(128) if norm else None)
    return x


def cuda(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def close(x, ref, tol, what):
    x = x.detach().cpu().double()
    bad = ((x - ref).abs() > 1.05 * tol + 1e-30) | ~torch.isfinite(x)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                           f"{float(((x - ref).abs() / (tol + 1e-30)).max()):.2f} of it")


def check(gdn, x, axis=None, interleaved=False, bwd=True):
    d = cuda(x)
    how = dict(q_weight=d["wq"], k_weight=d["wk"], eps=EPS, pair_axis=axis, interleaved=interleaved)
    freq = d["freq"] if x["freq"].numel() else None
    pos = d["pos"] if freq is not None else None
    angle = ops.angles(x["pos"], x["freq"], axis)
    q, k = gdn.rope_fwd(d["q"], d["k"], pos, freq, **how)
    close(q, *ops.rope(x["q"], x["wq"], angle, interleaved, EPS), "q")
    close(k, *ops.rope(x["k"], x["wk"], angle, interleaved, EPS), "k")
    if not bwd:
        return
    got = gdn.rope_bwd(d["q"], d["k"], pos, freq, d["gq"], d["gk"], **how)
    for name, dx, dw in (("q", got[0], got[2]), ("k", got[1], got[3])):
        rx, tx, rw, tw = ops.rope_bwd(x[name], x["w" + name], angle, interleaved, EPS, x["g" + name])
        close(dx, rx, tx, "d" + name)
        if rw is None:
            assert dw is None
        else:
            close(dw, rw, tw, "d weight of " + name)


@pytest.mark.parametrize("n,Hq,Hk", [(1, 1, 1), (1, 16, 4), (2, 3, 1), (77, 16, 4), (33, 6, 2), (130, 2, 2), (5, 100, 50),
                                     (1031, 4, 1)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes(gdn_lib, n, Hq, Hk, interleaved):
    check(gdn_lib, make(n, Hq, Hk, 64, seed=n + Hq), interleaved=interleaved)


@pytest.mark.parametrize("pairs", [0, 8, 16, 48, 56, 64])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
def test_parts_of_a_head(gdn_lib, pairs, norm, interleaved):
    check(gdn_lib, make(19, 4, 2, pairs, seed=pairs, norm=norm), interleaved=interleaved)


def test_one_of_the_norms(gdn_lib):
    x = make(40, 4, 2, 64, seed=5)
    check(gdn_lib, dict(x, wq=None))
    check(gdn_lib, dict(x, wk=None))


def test_rows_that_are_not_read(gdn_lib):
    """Without its weight a part's rows are not read in the backward, and may be left out in C."""
    d = cuda(make(40, 4, 2, 64, seed=5))
    want = gdn_lib.rope_bwd(d["q"], d["k"], d["pos"], d["freq"], d["gq"], d["gk"], q_weight=d["wq"])
    got = [torch.empty_like(t) for t in want[:3]]
    ws = torch.empty(gdn_lib.rope_workspace_bytes(40, 4, 2), dtype=torch.uint8, device="cuda")
    p = lambda t: t.data_ptr()
    rc = gdn_lib.lib().gdn_rope_bwd(p(d["q"]), None, p(d["wq"]), None, p(d["pos"]), p(d["freq"]), None, p(d["gq"]), p(d["gk"]),
                                    p(got[0]), p(got[1]), p(got[2]), None, 40, 4, 2, 128, 1, 64, 0, EPS, 512, 256, 512, 256, 512,
                                    256, p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_infinities_stay_where_they_are(gdn_lib):
    """What is not turned passes as it is, and an infinity reaches its pair alone."""
    x = make(6, 2, 1, 32, seed=6, norm=False)
    x["q"][2, 1, 100], x["q"][3, 0, 7] = float("inf"), float("-inf")
    d = cuda(x)
    q, _ = gdn_lib.rope_fwd(d["q"], d["k"], d["pos"], d["freq"])
    assert torch.equal(q[..., 64:], d["q"][..., 64:])
    bad = ~torch.isfinite(q[..., :64])
    where = torch.zeros_like(bad)
    where[3, 0, 7] = where[3, 0, 39] = True
    assert not (bad & ~where).any()


@pytest.mark.parametrize("axis", [(0,) * 16 + (1,) * 24 + (2,) * 24, tuple(j % 3 for j in range(64)), (1,) * 64])
@pytest.mark.parametrize("interleaved", [False, True])
def test_several_axes(gdn_lib, axis, interleaved):
    check(gdn_lib, make(57, 4, 2, 64, seed=6, axes=3), axis=axis, interleaved=interleaved)


@pytest.mark.parametrize("far", [10 ** 6, 2 ** 31 - 4100, -2 ** 31 + 10])
def test_far_positions(gdn_lib, far):
    """The angle keeps its fraction of a turn: at 2^31 an angle in fp32 would be off by tens of turns.
    (The 64-bit product of the definition is itself right to 2^-52 of the angle, 5e-7.)"""
    check(gdn_lib, make(64, 2, 1, 64, seed=7, far=far))


def test_frequencies_of_any_size(gdn_lib):
    x = make(50, 2, 1, 64, seed=8)
    x["freq"] = torch.cat([-x["freq"][:32], torch.tensor([0.0, 1e-30, 7.0, 100.5]), x["freq"][36:]])
    check(gdn_lib, x)


def test_many_rows(gdn_lib):
    """More tokens than the backward has blocks for."""
    check(gdn_lib, make(20011, 3, 1, 64, seed=9))


def test_zero_rows_and_tiny_values(gdn_lib):
    x = make(20, 2, 1, 64, seed=10)
    x["q"][3] = 0
    x["k"][4] = 1e-20
    check(gdn_lib, x)


def test_empty(gdn_lib):
    x = cuda(make(0, 2, 1, 64, seed=11))
    how = dict(q_weight=x["wq"], k_weight=x["wk"])
    q, k = gdn_lib.rope_fwd(x["q"], x["k"], x["pos"], x["freq"], **how)
    assert q.shape == (0, 2, 128) and k.shape == (0, 1, 128)
    dq, dk, dwq, dwk = gdn_lib.rope_bwd(x["q"], x["k"], x["pos"], x["freq"], x["gq"], x["gk"], **how)
    assert not dwq.any() and not dwk.any() and dq.shape[0] == 0


@pytest.mark.parametrize("shift", [0, 8])
def test_parts_of_one_buffer_in_place_and_batched(gdn_lib, shift):
    """q, k, v as parts of a projection's rows, turned where they lie; other columns keep what they hold."""
    B, T, Hq, Hk = 2, 37, 4, 2
    x = make(B * T, Hq, Hk, 64, seed=12)
    wide = torch.full((B, T, (Hq + 2 * Hk) * 128 + 2 * shift), 7.0).bfloat16()
    wide[..., shift:wide.shape[-1] - shift] = torch.cat([x[n].flatten(1) for n in "qkv"], 1).view(B, T, -1)
    wide = wide.cuda()
    q, k, v = (t.unflatten(-1, (-1, 128)) for t in
               wide[..., shift:wide.shape[-1] - shift].split([Hq * 128, Hk * 128, Hk * 128], 2))
    how = dict(q_weight=x["wq"].cuda(), k_weight=x["wk"].cuda(), eps=EPS)
    pos, freq = x["pos"].cuda().view(B, T), x["freq"].cuda()
    plain = gdn_lib.rope_fwd(q, k, pos, freq, **how)
    dplain = gdn_lib.rope_bwd(q, k, pos, freq, x["gq"].cuda().view(B, T, Hq, 128), x["gk"].cuda().view(B, T, Hk, 128), **how)
    # the backward in place of its cotangents
    gq, gk = x["gq"].cuda().view(B, T, Hq, 128), x["gk"].cuda().view(B, T, Hk, 128)
    din = gdn_lib.rope_bwd(q, k, pos, freq, gq, gk, dq=gq, dk=gk, **how)
    assert din[0] is gq and all(torch.equal(a, b) for a, b in zip(dplain, din))
    before = wide.clone()
    got = gdn_lib.rope_fwd(q, k, pos, freq, q_out=q, k_out=k, **how)
    assert got[0] is q and torch.equal(q, plain[0]) and torch.equal(k, plain[1])
    keep = torch.ones(wide.shape[-1], dtype=torch.bool)
    keep[shift:shift + (Hq + Hk) * 128] = False
    assert torch.equal(wide[..., keep], before[..., keep])
    angle = ops.angles(x["pos"], x["freq"])
    close(q.flatten(0, 1), *ops.rope(x["q"], x["wq"], angle, False, EPS), "q")


def test_gradients_against_differences(gdn_lib):
    """The forward's change along a direction against the gradients.  Outputs are rounded to bf16 (off by
    at most 2^-8 of each value), so a step of 1/4 is taken of a forward without norms, which is linear:
    the difference is then off by 2^-8 (|y1| + |y0|) |g| in sum at most, and by the gradient's own bound."""
    x = make(30, 2, 1, 64, seed=13, norm=False)
    d = cuda(x)
    dx = (torch.randn(30, 2, 128, generator=torch.Generator().manual_seed(14)) / 4).bfloat16().cuda()
    moved = (d["q"].float() + dx.float()).bfloat16()
    step = moved.double() - d["q"].double()
    y1, _ = gdn_lib.rope_fwd(moved, d["k"], d["pos"], d["freq"])
    y0, _ = gdn_lib.rope_fwd(d["q"], d["k"], d["pos"], d["freq"])
    dq, _, _, _ = gdn_lib.rope_bwd(d["q"], d["k"], d["pos"], d["freq"], d["gq"], d["gk"])
    g = d["gq"].double()
    change = float(((y1.double() - y0.double()) * g).sum())
    off = float((2.0 ** -8 * (y1.double().abs() + y0.double().abs()) * g.abs()).sum() +
                (2.0 ** -8 * dq.double().abs() * step.abs()).sum())
    assert abs(change - float((dq.double() * step).sum())) <= 1.05 * off


def test_repeated_calls_are_equal(gdn_lib):
    d = cuda(make(3000, 5, 5, 64, seed=15))
    how = dict(q_weight=d["wq"], k_weight=d["wk"])
    runs = [gdn_lib.rope_bwd(d["q"], d["k"], d["pos"], d["freq"], d["gq"], d["gk"], **how) for _ in range(2)]
    assert all(torch.equal(a, b) for a, b in zip(*runs))


# ---- into pages ---------------------------------------------------------------------------
def layout(kind, P, page, Hk):
    """A cache of the given memory order, as [P, page, Hk, 128], filled with a pattern."""
    fill = lambda *s: (torch.arange(torch.Size(s).numel()).view(s) % 251).bfloat16().cuda()
    if kind == "rows":
        return fill(P, page, Hk, 128), fill(P, page, Hk, 128)
    if kind == "heads":      # a head's rows of a page together
        return fill(P, Hk, page, 128).transpose(1, 2), fill(P, Hk, page, 128).transpose(1, 2)
    both = fill(P, 2, page, Hk, 136)[..., :128]  # keys and values of a page together, rows with a gap
    return both[:, 0], both[:, 1]


@pytest.mark.parametrize("kind", ["rows", "heads", "both"])
@pytest.mark.parametrize("n,page,Hq,Hk", [(1, 16, 4, 2), (50, 48, 6, 3), (300, 64, 2, 1)])
def test_append(gdn_lib, kind, n, page, Hq, Hk):
    x = make(n, Hq, Hk, 64, seed=n)
    d = cuda(x)
    P = n // page + 3
    kp, vp = layout(kind, P, page, Hk)
    gen = torch.Generator().manual_seed(n)
    slots = torch.randperm(P * page, generator=gen)[:n].int()
    if n > 4:
        slots[1], slots[3], slots[4] = -1, P * page, 2 ** 31 - 1     # padded tokens
    wantk, wantv = kp.clone(), vp.clone()
    plain = gdn_lib.rope_fwd(d["q"], d["k"], d["pos"], d["freq"], q_weight=d["wq"], k_weight=d["wk"])
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < P * page:
            wantk[s // page, s % page], wantv[s // page, s % page] = plain[1][t], d["v"][t]
    q = gdn_lib.rope_append(d["q"], d["k"], d["v"], d["pos"], d["freq"], kp, vp, slots.cuda(), q_weight=d["wq"],
                            k_weight=d["wk"])
    assert torch.equal(q, plain[0]) and torch.equal(kp, wantk) and torch.equal(vp, wantv)


def test_append_without_norm_or_rotation(gdn_lib):
    """Keys and values as they are."""
    d = cuda(make(20, 2, 2, 64, seed=21))
    kp, vp = layout("rows", 2, 16, 2)
    slots = torch.arange(20, dtype=torch.int32).cuda()
    q = gdn_lib.rope_append(d["q"], d["k"], d["v"], None, None, kp, vp, slots)
    assert torch.equal(q, d["q"]) and torch.equal(kp.view(32, 2, 128)[:20], d["k"])
    assert torch.equal(vp.view(32, 2, 128)[:20], d["v"])


def test_append_past_32_bit_offsets(gdn_lib):
    P, page, Hk = 9000, 256, 8     # 2.4e9 elements to a tensor, 4.7 GB
    kp = torch.zeros(P, page, Hk, 128, dtype=torch.bfloat16, device="cuda")
    d = cuda(make(3, 8, 8, 64, seed=22))
    slots = torch.tensor([0, P * page - 1, 8500 * page + 17], dtype=torch.int32).cuda()
    gdn_lib.rope_append(d["q"], d["k"], d["v"], d["pos"], d["freq"], kp, kp.clone(), slots, q_weight=d["wq"],
                        k_weight=d["wk"])
    _, k = gdn_lib.rope_fwd(d["q"], d["k"], d["pos"], d["freq"], q_weight=d["wq"], k_weight=d["wk"])
    assert torch.equal(kp.view(-1, Hk, 128)[slots.long()], k)
    assert int(kp.view(-1, Hk * 128).any(1).sum()) == 3
