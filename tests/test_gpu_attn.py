"""Causal attention over packed sequences against its 64-bit definition.

Tolerances, element by element (oracle.ops.attn gives them with the values): p
and ds are rounded once to bf16 (unit roundoff 2^-8 of each term of the sums they
enter), each result once more, delta = dO . o takes the rounded o; scores are fp32
sums of 128 products, off by at most 136 * 2^-23 of the sum of their sizes.
"""
import pytest
import torch

from oracle import ops

pytestmark = pytest.mark.gpu


def make(ql, kl, Hq, Hk, seed, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen).bfloat16()
    return dict(q=(r(sum(ql), Hq, 128).float() * spread).bfloat16(), k=r(sum(kl), Hk, 128), v=r(sum(kl), Hk, 128),
                dO=r(sum(ql), Hq, 128))


def cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def close(x, ref, tol, what):
    x = x.detach().cpu().double()
    none = ref == -float("inf")
    assert torch.equal(x[none], ref[none]), f"{what}: rows that see no key"
    x, ref, tol = x[~none], ref[~none], tol[~none]
    bad = ((x - ref).abs() > 1.05 * tol + 1e-30) | ~torch.isfinite(x)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                           f"{float(((x - ref).abs() / (tol + 1e-30)).max()):.2f} of it")


def eps_of(x, scale):
    """Scores are off by at most 136 * 2^-23 of the largest sum of sizes."""
    size = x["q"].float().norm(dim=-1).max() * x["k"].float().norm(dim=-1).max() if x["k"].numel() and x["q"].numel() else 0.0
    return float(scale * size * 136 * 2.0 ** -23)


def check(gdn, x, ql, kl, scale=None, bwd=True, most=None):
    sc = 128 ** -0.5 if scale is None else scale
    d = {n: t.cuda() for n, t in x.items()}
    args = dict(cu_q=cu(ql), cu_k=cu(kl), scale=scale)
    o, lse = gdn.attn_fwd(d["q"], d["k"], d["v"], max_q=max(ql), max_k=max(kl) if most is None else most, **args)
    k0 = cu(kl).tolist()[:-1]
    r = ops.attn(x["q"], x["k"], x["v"], ql, k0, kl, sc, x["dO"] if bwd else None, eps_of(x, sc))
    close(o, r["o"], r["o_tol"], "o")
    close(lse, r["lse"], r["lse_tol"], "lse")
    if bwd:
        got = gdn.attn_bwd(d["q"], d["k"], d["v"], o, lse, d["dO"], **args)
        for n, g in zip(("dq", "dk", "dv"), got):
            close(g, r[n], r[n + "_tol"], n)


CASES = [
    # queries, keys, heads
    ([1], [1], 1, 1), ([128], [128], 1, 1), ([129], [129], 2, 1), ([300, 1, 77, 0, 256], None, 4, 2),
    ([513], [513], 3, 1), ([100, 260], [100, 260], 6, 2),            # groups of 3: 126 rows to a tile
    ([64, 130], [700, 131], 8, 2),                                   # continuing cached keys
    ([50, 200, 3], [20, 130, 0], 4, 2),                              # more queries than keys: rows that see none
    ([0, 0], [5, 300], 2, 1),                                        # keys that no query sees
    ([40], [333], 16, 1), ([9], [260], 128, 1), ([7], [140], 100, 1),
]


@pytest.mark.parametrize("ql,kl,Hq,Hk", CASES)
def test_packed_sequences(gdn_lib, ql, kl, Hq, Hk):
    kl = ql if kl is None else kl
    check(gdn_lib, make(ql, kl, Hq, Hk, seed=sum(ql) + Hq), ql, kl)


@pytest.mark.parametrize("scale,spread", [(1.0, 1.0), (0.02, 1.0), (None, 8.0)])
def test_sharp_and_flat_rows(gdn_lib, scale, spread):
    """Rows that one key takes whole (the running maximum rises often), and nearly even ones."""
    check(gdn_lib, make([400], [400], 2, 1, seed=3, spread=spread), [400], [400], scale=scale)


@pytest.mark.parametrize("rows,cap,Hq,Hk", [(1, 3000, 1, 1), (3, 5000, 8, 2), (5, 2500, 6, 2), (2, 4000, 16, 16)])
@pytest.mark.parametrize("tokens", [1, 4])
def test_tokens_over_a_cache(gdn_lib, rows, cap, Hq, Hk, tokens):
    """Caches of one capacity, filled to different lengths; what lies past them is NaN."""
    gen = torch.Generator().manual_seed(rows + Hq)
    used = [max(tokens, int(torch.randint(1, cap + 1, (1,), generator=gen))) for _ in range(rows)]
    used[0] = cap
    ql = [tokens] * rows
    x = make(ql, [cap] * rows, Hq, Hk, seed=11)
    for n in ("k", "v"):
        c = x[n].view(rows, cap, Hk, 128)
        for b, m in enumerate(used):
            c[b, m:] = float("nan")
    d = {n: t.cuda() for n, t in x.items()}
    klen = torch.tensor(used, dtype=torch.int32).cuda()
    clean = {n: torch.nan_to_num(t) for n, t in x.items()}
    r = ops.attn(x["q"], clean["k"], clean["v"], ql, [b * cap for b in range(rows)], used, 128 ** -0.5,
                 eps=eps_of(clean, 128 ** -0.5))
    for most in (cap, 1):  # max_k only steers the split
        o, lse = gdn_lib.attn_fwd(d["q"], d["k"], d["v"], cu_q=cu(ql), cu_k=cu([cap] * rows), k_len=klen, max_k=most)
        close(o, r["o"], r["o_tol"], "o")
        close(lse, r["lse"], r["lse_tol"], "lse")
    shape = lambda t, n: t.view(rows, n, -1, 128)
    o, lse = gdn_lib.attn_fwd(shape(d["q"], tokens), shape(d["k"], cap), shape(d["v"], cap), k_len=klen)
    close(o.flatten(0, 1), r["o"], r["o_tol"], "o (batched layout)")


def test_parts_of_one_buffer_batched_layout(gdn_lib):
    B, T, Hq, Hk = 2, 200, 4, 2
    x = make([T] * B, [T] * B, Hq, Hk, seed=12)
    qkv = torch.cat([x[n].flatten(1) for n in ("q", "k", "v")], 1).cuda().view(B, T, -1)
    q, k, v = qkv.split([Hq * 128, Hk * 128, Hk * 128], 2)
    q, k, v = q.view(B, T, Hq, 128), k.view(B, T, Hk, 128), v.view(B, T, Hk, 128)
    o, lse = gdn_lib.attn_fwd(q, k, v)
    r = ops.attn(x["q"], x["k"], x["v"], [T] * B, [0, T], [T] * B, 128 ** -0.5, x["dO"], eps_of(x, 128 ** -0.5))
    close(o.flatten(0, 1), r["o"], r["o_tol"], "o")
    got = gdn_lib.attn_bwd(q, k, v, o, lse, x["dO"].cuda().view(B, T, Hq, 128))
    for n, g in zip(("dq", "dk", "dv"), got):
        close(g.flatten(0, 1), r[n], r[n + "_tol"], n)


def test_neighbouring_sequences_do_not_matter(gdn_lib):
    ql = [130, 90, 200]
    x = make(ql, ql, 4, 2, seed=13)
    d = {n: t.clone().cuda() for n, t in x.items()}
    for t in d.values():
        t[130:220] = float("nan")
        t[140:150] = float("inf")
    keep = [i for i in range(420) if not 130 <= i < 220]
    y = {n: t[keep] for n, t in x.items()}
    r = ops.attn(y["q"], y["k"], y["v"], [130, 200], [0, 130], [130, 200], 128 ** -0.5, y["dO"], eps_of(y, 128 ** -0.5))
    args = dict(cu_q=cu(ql), cu_k=cu(ql))
    o, lse = gdn_lib.attn_fwd(d["q"], d["k"], d["v"], **args)
    close(o[keep], r["o"], r["o_tol"], "o")
    got = gdn_lib.attn_bwd(d["q"], d["k"], d["v"], o, lse, d["dO"], **args)
    for n, g in zip(("dq", "dk", "dv"), got):
        close(g[keep], r[n], r[n + "_tol"], n)


def test_no_queries_or_no_keys(gdn_lib):
    x = {n: t.cuda() for n, t in make([0, 0], [3, 4], 2, 1, seed=14).items()}
    o, lse = gdn_lib.attn_fwd(x["q"], x["k"], x["v"], cu_q=cu([0, 0]), cu_k=cu([3, 4]))
    assert o.shape == (0, 2, 128) and lse.shape == (0, 2)
    dq, dk, dv = gdn_lib.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], cu_q=cu([0, 0]), cu_k=cu([3, 4]))
    assert not dk.any() and not dv.any()
    x = {n: t.cuda() for n, t in make([3, 4], [0, 0], 2, 1, seed=15).items()}
    o, lse = gdn_lib.attn_fwd(x["q"], x["k"], x["v"], cu_q=cu([3, 4]), cu_k=cu([0, 0]))
    assert not o.any() and bool((lse == -float("inf")).all())
    dq, dk, dv = gdn_lib.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], cu_q=cu([3, 4]), cu_k=cu([0, 0]))
    assert not dq.any() and dk.shape[0] == 0


def test_repeated_calls_are_equal(gdn_lib):
    x = {n: t.cuda() for n, t in make([700, 129], [700, 129], 4, 2, seed=16).items()}
    args = dict(cu_q=cu([700, 129]), cu_k=cu([700, 129]))
    runs = []
    for _ in range(2):
        o, lse = gdn_lib.attn_fwd(x["q"], x["k"], x["v"], **args)
        runs.append((o, lse) + gdn_lib.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["dO"], **args))
    assert all(torch.equal(a, b) for a, b in zip(*runs))
