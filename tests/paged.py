"""Caches in pages for the tests: random pages, tables in random order, and what must not matter made NaN."""
import torch


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32)


def cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)


def cache(ql, kl, Hq, Hk, page, seed, spare=2, spread=1.0, wide=0, nan=True):
    """q, k_pages, v_pages, table and lengths of sequences of ql new tokens and kl keys in all, on the
    host.  Rows behind a sequence's keys and spare pages are NaN."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    need = [-(-m // page) for m in kl]
    P = sum(need) + spare
    order = torch.randperm(P, generator=gen)
    table = torch.full((len(kl), max(need + [0]) + wide), -7, dtype=torch.int32)
    kp, vp = r(P, page, Hk, 128).bfloat16(), r(P, page, Hk, 128).bfloat16()
    at = 0
    used = torch.zeros(P, page, dtype=torch.bool)
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m].int()
        at += m
        for i in range(m):
            used[table[s, i], :min(page, kl[s] - i * page)] = True
    if nan:
        kp[~used], vp[~used] = float("nan"), float("nan")
    return dict(q=(spread * r(sum(ql), Hq, 128)).bfloat16(), kp=kp, vp=vp, table=table, k_len=ints(kl), cu=cu(ql),
                weights=torch.rand(P, Hk, page, generator=gen) * 3)


def cuda(x):
    return {n: t.cuda() for n, t in x.items()}
