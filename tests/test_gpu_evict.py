"""Eviction of the lightest keys of a paged cache against a plain sort: what moves is copied, so equal bits."""
import pytest
import torch

import paged
from oracle import ops

pytestmark = pytest.mark.gpu


def same(a, b):
    """Equal bits, NaN included."""
    view = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.cpu().contiguous().view(view), b.cpu().contiguous().view(view))


def check(gdn, x, kl, budget, recent, to=None, d=None):
    d = paged.cuda(x) if d is None else d
    want = ops.cache_evict(x["kp"], x["vp"], x["weights"], x["table"], kl, budget, recent, x["table"] if to is None else to)
    kp, vp, w = d["kp"], d["vp"], d["weights"]
    n = gdn.cache_evict(kp, vp, w, d["table"], d["k_len"], budget, recent=recent, to_table=None if to is None else to.cuda())
    assert n.tolist() == want[3]
    assert same(w, want[2]) and same(kp, want[0]) and same(vp, want[1])
    return want[3]


def weights(x, seed, kind):
    gen = torch.Generator().manual_seed(seed)
    r = torch.randn(x["weights"].shape, generator=gen)
    if kind == "spread":
        x["weights"] = torch.exp(4 * r)
    elif kind == "ties":
        x["weights"] = (r * 2).round().abs()
    elif kind == "equal":
        x["weights"] = torch.ones_like(r)
    elif kind == "signs":            # any numbers at all, both zeros among them
        x["weights"] = torch.where(r.abs() < 0.3, torch.where(r > 0, 0.0, -0.0), r * 1e30)
    elif kind == "special":
        x["weights"] = torch.where(r > 1.2, float("inf"), torch.where(r < -1.2, float("nan"), torch.where(r.abs() < 0.2, -float("inf"), r)))
    elif kind == "low bits":         # ranks that differ in their last bits alone
        x["weights"] = (1.0 + (r.abs() * 40).floor() * 2.0 ** -23).float()
    return x


KINDS = ["spread", "ties", "equal", "signs", "special", "low bits"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kl,Hk,page,budget,recent", [
    ([100], 1, 16, 40, 10), ([100, 0, 1, 39, 40, 41], 2, 16, 40, 10), ([300, 257], 3, 48, 64, 0),
    ([500, 20], 2, 64, 128, 128), ([500, 20], 2, 64, 128, 1000), ([90], 2, 32, 0, 5), ([90], 2, 32, 1, 0), ([1100, 64], 1, 256, 1000, 1),
])
@pytest.mark.parametrize("elsewhere", [False, True])
def test_budgets(gdn_lib, kind, kl, Hk, page, budget, recent, elsewhere):
    need = -(-min(budget, max(kl)) // page)
    x = weights(paged.cache([1] * len(kl), kl, Hk, Hk, page, seed=budget + len(kl), spare=need * len(kl) + 1), budget, kind)
    to = None
    if elsewhere:
        free = sorted(set(range(x["kp"].shape[0])) - set(x["table"].flatten().tolist()))
        # (as many target rows as the table could keep)
        wide = -(-min(budget, x["table"].shape[1] * page) // page)
        to = torch.full((len(kl), wide), -1, dtype=torch.int32)
        for s, m in enumerate(kl):
            for i in range(-(-min(m, budget) // page)):
                to[s, i] = free.pop()
    check(gdn_lib, x, kl, budget, recent, to)


@pytest.mark.parametrize("kind", ["spread", "ties"])
@pytest.mark.parametrize("kl,budget", [([5000, 3333], 2000), ([60000], 10000), ([50000, 49153], 49000)])
def test_long_caches(gdn_lib, kind, kl, budget):
    """Up to and beyond the weights that shared memory holds (49152), in place."""
    x = weights(paged.cache([1] * len(kl), kl, 1, 1, 256, seed=budget), budget, kind)
    check(gdn_lib, x, kl, budget, budget // 3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kl,Hk,page,budget,recent", [([9000, 4100, 3], 2, 64, 3000, 1000), ([20001], 1, 48, 777, 0),
                                                      ([16500, 40000], 1, 16, 16000, 15990)])
def test_lists_of_several_blocks(gdn_lib, kind, kl, Hk, page, budget, recent):
    """Caches whose keys are shared out, ties and the last ones across the cuts."""
    x = weights(paged.cache([1] * len(kl), kl, Hk, Hk, page, seed=budget), budget, kind)
    check(gdn_lib, x, kl, budget, recent)


@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_short_sequences_of_a_wide_table(gdn_lib, kind):
    """A table for 65536 keys and few of them there: most of the blocks have none."""
    kl = [300, 0, 130, 2500]
    x = weights(paged.cache([1] * 4, kl, 1, 1, 64, seed=3, wide=1000), 3, kind)
    check(gdn_lib, x, kl, 120, 20)


def test_many_long_lists(gdn_lib):
    """More keys than shared memory holds, in more lists than are shared out: 80 over the same pages."""
    n, m, budget = 20, 49300, 16
    x = weights(paged.cache([1], [m], 4, 4, 64, seed=12, spare=n), 12, "ties")
    free = sorted(set(range(x["kp"].shape[0])) - set(x["table"].flatten().tolist()))
    x["table"] = x["table"].repeat(n, 1)
    kl = [m - 3 * s for s in range(n)]
    x["k_len"] = paged.ints(kl)
    check(gdn_lib, x, kl, budget, 5, torch.tensor([[f] for f in free[:n]], dtype=torch.int32))


def test_nothing_to_drop_leaves_everything(gdn_lib):
    x = paged.cache([1, 1], [77, 33], 2, 2, 16, seed=4)
    d = paged.cuda(x)
    n = gdn_lib.cache_evict(d["kp"], d["vp"], d["weights"], d["table"], d["k_len"], 1000, recent=7)
    assert n.tolist() == [77, 33] and same(d["kp"], x["kp"]) and same(d["vp"], x["vp"]) and same(d["weights"], x["weights"])


@pytest.mark.parametrize("recent", [0, 50])
def test_absent_pages(gdn_lib, recent):
    """Keys on absent pages never stay, and take no part of the budget."""
    x = weights(paged.cache([1, 1], [200, 90], 2, 2, 16, seed=5), 5, "spread")
    x["table"][0, 7], x["table"][0, 12], x["table"][1, 5] = -1, x["kp"].shape[0], 2 ** 31 - 1
    check(gdn_lib, x, [200, 90], 60, recent)


def test_target_pages_that_are_absent(gdn_lib):
    x = weights(paged.cache([1], [100], 2, 2, 16, seed=6, spare=5), 6, "spread")
    free = sorted(set(range(x["kp"].shape[0])) - set(x["table"].flatten().tolist()))
    check(gdn_lib, x, [100], 50, 8, torch.tensor([[free[0], -1, free[1], 10 ** 6]], dtype=torch.int32))


@pytest.mark.parametrize("kind", ["heads", "both"])
def test_layouts(gdn_lib, kind):
    x = weights(paged.cache([1, 1], [300, 41], 3, 3, 32, seed=7), 7, "spread")
    d = paged.cuda(x)
    if kind == "heads":
        d["kp"], d["vp"] = (d[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("kp", "vp"))
    else:
        one = torch.stack([d["kp"], d["vp"]], 1).contiguous()
        d["kp"], d["vp"] = one[:, 0], one[:, 1]
    check(gdn_lib, x, [300, 41], 100, 20, d=d)


def test_the_table_named_as_target_is_in_place(gdn_lib):
    x = weights(paged.cache([1], [500], 2, 2, 16, seed=8), 8, "spread")
    d = paged.cuda(x)
    want = ops.cache_evict(x["kp"], x["vp"], x["weights"], x["table"], [500], 300, 20, x["table"])
    n = gdn_lib.cache_evict(d["kp"], d["vp"], d["weights"], d["table"], d["k_len"], 300, recent=20, to_table=d["table"])
    assert n.tolist() == want[3] and same(d["kp"], want[0]) and same(d["vp"], want[1]) and same(d["weights"], want[2])


def test_lengths_beyond_the_table(gdn_lib):
    x = weights(paged.cache([1, 1], [64, 64], 2, 2, 16, seed=9), 9, "spread")
    d = paged.cuda(x)
    d["k_len"] = torch.tensor([1 << 30, -3], dtype=torch.int32).cuda()
    check(gdn_lib, x, [64, 0], 30, 4, d=d)


def test_no_pages(gdn_lib):
    e = torch.zeros(0, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    n = gdn_lib.cache_evict(e, e, torch.zeros(0, 2, 16, device="cuda"), torch.zeros(2, 0, dtype=torch.int32, device="cuda"),
                            torch.tensor([5, 0], dtype=torch.int32).cuda(), 4)
    assert n.tolist() == [0, 0]
