"""Attention of new tokens over a paged cache, and the weight that each key receives, against their
64-bit definitions (bounds: oracle.ops.attn_paged, attn_paged_weights)."""
import pytest
import torch

import paged
from oracle import ops
from test_gpu_attn import close

pytestmark = pytest.mark.gpu


def eps_of(x, scale):
    """Scores are off by at most 136 * 2^-23 of the largest sum of sizes."""
    k = torch.nan_to_num(x["kp"].float())
    if not x["q"].numel() or not k.numel():
        return 0.0
    return float(scale * x["q"].float().norm(dim=-1).max() * k.norm(dim=-1).max() * 136 * 2.0 ** -23)


def both(gdn, x, ql, kl, scale=None, most=None, weights=True, d=None, most_q="exact"):
    sc = 128 ** -0.5 if scale is None else scale
    d = paged.cuda(x) if d is None else d
    args = dict(cu_q=d["cu"], max_q=max(ql + [0]) if most_q == "exact" else most_q, max_k=most, scale=scale)
    o, lse = gdn.attn_paged(d["q"], d["kp"], d["vp"], d["table"], d["k_len"], **args)
    eps = eps_of(x, sc)
    r = ops.attn_paged(x["q"], x["kp"], x["vp"], x["table"], ql, kl, sc, eps)
    close(o, r["o"], r["o_tol"], "o")
    close(lse, r["lse"], r["lse_tol"], "lse")
    if weights:
        w = d["weights"].clone()
        assert gdn.attn_paged_weights(d["q"], d["kp"], lse, d["table"], d["k_len"], w, **args) is w
        want, tol = ops.attn_paged_weights(x["q"], x["kp"], lse.cpu(), x["table"], ql, kl, x["weights"], sc, eps)
        close(w, want, tol, "weights")
        same = tol <= 2.0 ** -22 * x["weights"].double().abs()   # (places that nothing was added to)
        assert torch.equal(w.cpu()[same], x["weights"][same])
    return o, lse


CASES = [
    # new tokens, keys, heads
    ([1], [1], 1, 1), ([1], [16], 4, 1), ([1], [17], 4, 2), ([128], [128], 1, 1), ([129], [129], 2, 1),
    ([300, 1, 77, 0, 256], [300, 1, 77, 0, 256], 4, 2),
    ([513], [700], 3, 1), ([100, 260], [100, 1260], 6, 2),           # groups of 3: 126 rows to a tile
    ([64, 130, 3], [2700, 131, 3], 8, 2),                            # continuing cached keys
    ([50, 200, 3], [20, 130, 0], 4, 2),                              # more queries than keys: rows that see none
    ([0, 0], [5, 300], 2, 1), ([0, 2], [40, 0], 2, 1), ([0, 3], [0, 0], 8, 2), ([200], [0], 4, 2),  # (no table at all)
    ([40], [333], 16, 1), ([9], [260], 128, 1), ([7], [140], 100, 1),
    ([1, 1, 1, 2, 1], [4000, 1, 0, 129, 2048], 8, 2), ([1] * 40, list(range(0, 400, 10)), 4, 4),
]


@pytest.mark.parametrize("ql,kl,Hq,Hk", CASES)
@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_chunks_over_pages(gdn_lib, ql, kl, Hq, Hk, page):
    x = paged.cache(ql, kl, Hq, Hk, page, seed=sum(kl) + Hq + page, wide=page % 3)
    both(gdn_lib, x, ql, kl, most=max(kl))


@pytest.mark.parametrize("ql,kl,Hq,Hk", [
    ([1300], [1300], 16, 8),                                         # pairs of CTAs with several key tiles each
    ([1100, 900], [1100, 3001], 16, 8), ([70] * 6, list(range(1990, 2014, 4)), 8, 2),   # CTAs with several
    ([400, 1, 64, 3, 65, 1, 0, 1], [500, 3000, 3000, 2900, 3000, 1, 7, 2800], 8, 4),    # long ones beside short ones
    ([64, 60, 65], [1000, 64, 2500], 4, 1), ([200, 1, 1, 1, 1, 1], [777, 500, 1, 0, 1111, 40], 8, 2),  # several query tiles
])
def test_several_tiles_each(gdn_lib, ql, kl, Hq, Hk):
    """CTAs that take one key tile, or one query tile, after another."""
    x = paged.cache(ql, kl, Hq, Hk, 32, seed=len(ql))
    both(gdn_lib, x, ql, kl, most=max(kl))


@pytest.mark.parametrize("page", [32, 80, 112, 128, 1024])
@pytest.mark.parametrize("most", [None, 1, 3000, 100000])
@pytest.mark.parametrize("most_q", [None, 1, 100000])
def test_bounds_only_steer(gdn_lib, page, most, most_q):
    """max_q and max_k, too small or too large, and page sizes with other powers of two."""
    for ql, kl in (([1, 2, 1], [2999, 1500, 17]), ([300, 5], [1300, 2000])):
        x = paged.cache(ql, kl, 4, 2, page, seed=page)
        both(gdn_lib, x, ql, kl, most=most, most_q=most_q)


@pytest.mark.parametrize("Hq,Hk", [(8, 8), (8, 2), (6, 2), (16, 1)])
def test_many_sequences_of_any_length(gdn_lib, Hq, Hk):
    """More items than are planned at a time, tokens and prompts and sequences without either, in any order."""
    gen = torch.Generator().manual_seed(Hq + Hk)
    n = 150
    ql = torch.where(torch.rand(n, generator=gen) < 0.7, 1, torch.randint(0, 90, (n,), generator=gen)).tolist()
    kl = [max(0, q + int(k)) for q, k in zip(ql, torch.randint(-40, 160, (n,), generator=gen))]
    kl[7], kl[90] = 3000, 0
    x = paged.cache(ql, kl, Hq, Hk, 16, seed=2)
    for most_q in (None, 1):
        both(gdn_lib, x, ql, kl, most_q=most_q, weights=most_q is None)


@pytest.mark.parametrize("n,most", [(33, 400), (64, 300), (1030, 20)])
def test_prompts_of_many_sequences(gdn_lib, n, most):
    """More sequences than a warp has lanes, a few of them long beside short ones."""
    gen = torch.Generator().manual_seed(n)
    ql = torch.randint(0, most, (n,), generator=gen).tolist()
    ql[n // 2], ql[n - 1] = 500, 1
    kl = [q + int(k) for q, k in zip(ql, torch.randint(0, 60, (n,), generator=gen))]
    x = paged.cache(ql, kl, 4, 1, 32, seed=n)
    both(gdn_lib, x, ql, kl, most=max(kl))


@pytest.mark.parametrize("scale,spread", [(1.0, 1.0), (0.02, 1.0), (None, 8.0)])
def test_sharp_and_flat_rows(gdn_lib, scale, spread):
    x = paged.cache([300], [700], 2, 1, 64, seed=3, spread=spread)
    both(gdn_lib, x, [300], [700], scale=scale)


@pytest.mark.parametrize("ql,kl", [([1, 1], [900, 300]), ([200, 130], [900, 130])])
@pytest.mark.parametrize("entry", [-1, 2 ** 31 - 1, "pages"])
def test_absent_pages(gdn_lib, ql, kl, entry):
    """Keys on pages outside the cache are seen by nobody; a row left without keys is empty."""
    page = 48
    x = paged.cache(ql, kl, 4, 2, page, seed=5)
    bad = x["kp"].shape[0] if entry == "pages" else entry
    x["table"][0, 0] = x["table"][0, 3] = x["table"][0, -1] = bad
    x["table"][1, :] = bad                       # the second sequence has none left
    o, lse = both(gdn_lib, x, ql, kl)
    assert not o[ql[0]:].any() and bool((lse[ql[0]:] == -float("inf")).all())


@pytest.mark.parametrize("ql,kl", [([1, 1, 4], [900, 300, 64]), ([200, 130, 4], [900, 130, 64])])
def test_shared_pages(gdn_lib, ql, kl):
    """Sequences with a common beginning in the same pages, and a table that names a page twice."""
    page = 32
    x = paged.cache(ql, kl, 4, 2, page, seed=6)
    x["table"][1, :4] = x["table"][0, :4]
    x["table"][2, :2] = x["table"][0, 0]
    both(gdn_lib, x, ql, kl)


@pytest.mark.parametrize("kind", ["heads", "both", "gaps"])
@pytest.mark.parametrize("ql,kl", [([1, 3], [500, 77]), ([140, 30], [140, 600])])
def test_layouts(gdn_lib, kind, ql, kl):
    Hq, Hk, page = 6, 3, 32
    x = paged.cache(ql, kl, Hq, Hk, page, seed=7)
    d = paged.cuda(x)
    P = d["kp"].shape[0]
    if kind == "heads":
        d["kp"], d["vp"] = (d[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("kp", "vp"))
    elif kind == "both":
        one = torch.stack([d["kp"], d["vp"]], 1).contiguous()
        d["kp"], d["vp"] = one[:, 0], one[:, 1]
    else:
        wide = torch.full((2, P, page, Hk, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[0, ..., :128], wide[1, ..., :128] = d["kp"], d["vp"]
        d["kp"], d["vp"] = wide[0, ..., :128], wide[1, ..., :128]
        qw = torch.full((sum(ql), Hq * 128 + 256), float("nan"), dtype=torch.bfloat16, device="cuda")
        qw[:, 128:-128] = d["q"].flatten(1)
        d["q"] = qw[:, 128:-128].unflatten(1, (Hq, 128))
        tw = torch.full((len(kl), d["table"].shape[1] + 5), -9, dtype=torch.int32, device="cuda")
        tw[:, 2:-3] = d["table"]
        d["table"] = tw[:, 2:-3]
    both(gdn_lib, x, ql, kl, d=d)


def test_batched_layout(gdn_lib):
    B, T = 3, 5
    kl = [400, 5, 33]
    x = paged.cache([T] * B, kl, 4, 2, 16, seed=8)
    d = paged.cuda(x)
    o, lse = gdn_lib.attn_paged(d["q"], d["kp"], d["vp"], d["table"], d["k_len"], cu_q=d["cu"])
    o2, lse2 = gdn_lib.attn_paged(d["q"].view(B, T, 4, 128), d["kp"], d["vp"], d["table"], d["k_len"])
    assert torch.equal(o, o2.flatten(0, 1)) and torch.equal(lse, lse2.flatten(0, 1))
    w, w2 = d["weights"].clone(), d["weights"].clone()
    gdn_lib.attn_paged_weights(d["q"], d["kp"], lse, d["table"], d["k_len"], w, cu_q=d["cu"])
    gdn_lib.attn_paged_weights(d["q"].view(B, T, 4, 128), d["kp"], lse2, d["table"], d["k_len"], w2)
    assert torch.equal(w, w2)


def test_lengths_beyond_the_table(gdn_lib):
    """A length past what the table covers is held there; a negative one is none."""
    x = paged.cache([2, 1], [64, 64], 2, 1, 32, seed=9)
    d = paged.cuda(x)
    d["k_len"] = torch.tensor([1000, -4], dtype=torch.int32).cuda()
    both(gdn_lib, x, [2, 1], [64, 0], d=d)


@pytest.mark.parametrize("ql,kl", [([1, 1], [700, 90]), ([150, 140], [700, 140])])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_scores_that_are_not_numbers(gdn_lib, ql, kl, value):
    """A key of NaN or infinity: the rows that see it are NaN, all others keep their value; its weights
    and those of the other keys that such rows see are NaN."""
    x = paged.cache(ql, kl, 4, 2, 16, seed=12)
    key = kl[0] - ql[0] // 2 - 1
    clean = {n: t.clone() for n, t in x.items()}
    x["kp"][x["table"][0, key // 16], key % 16, 1, 5] = value
    d = paged.cuda(x)
    o, lse = gdn_lib.attn_paged(d["q"], d["kp"], d["vp"], d["table"], d["k_len"], cu_q=d["cu"])
    r = ops.attn_paged(clean["q"], clean["kp"], clean["vp"], clean["table"], ql, kl, 128 ** -0.5, eps_of(clean, 128 ** -0.5))
    hit = torch.zeros(sum(ql), 4, dtype=torch.bool)
    for i in range(ql[0]):
        hit[i, 2:] = key <= i + kl[0] - ql[0]
    if value != value:   # (an infinity gives scores of both signs; those of minus infinity drop the key)
        assert bool(torch.isnan(o.cpu()[hit]).all()) and bool(torch.isnan(lse.cpu()[hit]).all())
    close(o.cpu()[~hit], r["o"][~hit], r["o_tol"][~hit], "o of the other rows")
    close(lse.cpu()[~hit], r["lse"][~hit], r["lse_tol"][~hit], "lse of the other rows")
    if value != value:
        w = gdn_lib.attn_paged_weights(d["q"], d["kp"], lse, d["table"], d["k_len"], d["weights"].clone(), cu_q=d["cu"])
        want, tol = ops.attn_paged_weights(clean["q"], clean["kp"], torch.where(hit, 0.0, lse.cpu()), clean["table"], ql,
                                           kl, clean["weights"], 128 ** -0.5, eps_of(clean, 128 ** -0.5))
        gone = torch.zeros_like(w.cpu(), dtype=torch.bool)
        for j in range(kl[0]):     # every key that a hit row sees
            gone[x["table"][0, j // 16], 1, j % 16] = True
        assert bool(torch.isnan(w.cpu()[gone]).all())
        close(w.cpu()[~gone], want[~gone], tol[~gone], "weights of the other head and sequence")


def test_rows_without_a_log_sum_add_nothing(gdn_lib):
    x = paged.cache([3], [70], 2, 1, 16, seed=13)
    d = paged.cuda(x)
    lse = torch.full((3, 2), -float("inf"), device="cuda")
    w = gdn_lib.attn_paged_weights(d["q"], d["kp"], lse, d["table"], d["k_len"], d["weights"].clone(), cu_q=d["cu"])
    assert torch.equal(w, d["weights"])


def test_pages_past_32_bit_offsets(gdn_lib):
    """Pages whose rows lie beyond 2^31 elements and bytes."""
    P, page, Hk = 9000, 256, 8
    gen = torch.Generator(device="cuda").manual_seed(14)
    kp = torch.zeros(P, page, Hk, 128, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.tensor([[8999, 3, 8500], [8200, 0, 1]], dtype=torch.int32)
    for e in table.flatten().tolist():
        kp[e], vp[e] = (torch.randn(page, Hk, 128, generator=gen, device="cuda").bfloat16() for _ in "kv")
    small = dict(q=torch.randn(2, 8, 128, generator=gen, device="cuda").bfloat16())
    k_len = torch.tensor([700, 300], dtype=torch.int32).cuda()
    w = torch.zeros(P, Hk, page, device="cuda")
    args = dict(cu_q=paged.cu([1, 1]).cuda())
    o, lse = gdn_lib.attn_paged(small["q"], kp, vp, table.cuda(), k_len, **args)
    gdn_lib.attn_paged_weights(small["q"], kp, lse, table.cuda(), k_len, w, **args)
    near = table.flatten().long()
    again = torch.arange(6, dtype=torch.int32).view(2, 3).cuda()
    k2, v2 = kp[near.cuda()], vp[near.cuda()]
    o2, lse2 = gdn_lib.attn_paged(small["q"], k2, v2, again, k_len, **args)
    w2 = gdn_lib.attn_paged_weights(small["q"], k2, lse2, again, k_len, torch.zeros(6, Hk, page, device="cuda"), **args)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(w[near.cuda()], w2)
    assert float(w.sum()) == pytest.approx(16.0, rel=1e-4)    # 2 tokens of 8 heads


def test_repeated_calls_are_equal(gdn_lib):
    for ql, kl in (([300, 1], [900, 500]), ([1, 2], [5000, 100])):
        d = paged.cuda(paged.cache(ql, kl, 4, 2, 16, seed=16))
        runs = []
        for _ in range(2):
            o, lse = gdn_lib.attn_paged(d["q"], d["kp"], d["vp"], d["table"], d["k_len"], cu_q=d["cu"])
            w = gdn_lib.attn_paged_weights(d["q"], d["kp"], lse, d["table"], d["k_len"], d["weights"].clone(), cu_q=d["cu"])
            runs.append((o, lse, w))
        assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_status_words(gdn_lib):
    """The workspaces' status words read clean after calls of each kernel."""
    for ql, kl in (([300, 1], [900, 500]), ([1, 2], [5000, 100])):
        d = paged.cuda(paged.cache(ql, kl, 4, 2, 16, seed=17))
        ws = torch.full((gdn_lib.attn_paged_workspace_bytes(2, sum(ql), d["table"].shape[1] * 16, 0, max(kl), 4, 2),), 255,
                        dtype=torch.uint8, device="cuda")
        o, lse = gdn_lib.attn_paged(d["q"], d["kp"], d["vp"], d["table"], d["k_len"], cu_q=d["cu"], max_k=max(kl), workspace=ws)
        assert gdn_lib.workspace_status(ws) == 0
        ws.fill_(255)
        gdn_lib.attn_paged_weights(d["q"], d["kp"], lse, d["table"], d["k_len"], d["weights"], cu_q=d["cu"], workspace=ws)
        assert gdn_lib.workspace_status(ws) == 0
