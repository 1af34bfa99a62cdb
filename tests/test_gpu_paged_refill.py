"""Calls whose CTAs have more items than are planned at a time, in both kernels over pages, against the
64-bit definitions.  (The number of items to a CTA is found by the plan's own arithmetic.)"""
import os
import re

import pytest
import torch

import paged
from test_gpu_paged import both
from test_paged_models import items, tiles

pytestmark = pytest.mark.gpu
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_rnn_gb300", "csrc")


def constant(name):
    with open(os.path.join(CSRC, "gdn_attn_paged.cu")) as f:
        return int(re.search(rf"\b{name} = (\d+)", f.read()).group(1))


def most_items(ql, kl, G, Hk, few):
    """Items of the run that has the most."""
    kind, S = ("FEW", 128 // G) if few else ("MANY", 2 * (128 // G))
    extra, narrow = constant(kind + "_EXTRA"), constant(kind + "_RUN")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    widths = [w for q, k in zip(ql, kl) for _ in range(Hk) for _, w in items(q, k, S, extra)]
    V, most = sum(widths), (2 if few else 1) * sms
    C = most if V >= narrow * most else max(1, V // narrow)
    begin = lambda c: V // C * c + min(c, V % C)
    count, c, pos = [0] * C, 0, 0
    for w in widths:
        while begin(c + 1) <= pos:
            c += 1
        d = c
        while d < C and begin(d) < pos + w:    # (an item that is cut counts where it has key tiles)
            x0, x1 = max(0, begin(d) - pos), min(w, begin(d + 1) - pos)
            count[d] += (x0 == 0 and x1 == w) or tiles(x0, w, extra) < tiles(x1, w, extra)
            d += 1
        pos += w
    return max(count)


def lengths(n, q, k, seed, long=()):
    """q: (least, most) new tokens; k: keys that were there, at most; long: (sequence, its keys)."""
    gen = torch.Generator().manual_seed(seed)
    ql = torch.randint(q[0], q[1] + 1, (n,), generator=gen).tolist()
    kl = [max(0, a + int(b)) for a, b in zip(ql, torch.randint(-2 if q[1] > 1 else 0, k + 1, (n,), generator=gen))]
    for s, m in long:
        kl[s] = m
    return ql, kl


@pytest.mark.parametrize("n,q,k,Hq,Hk,long", [
    (1024, (1, 1), 40, 8, 8, ()),                            # tokens of many users
    (1500, (1, 1), 20, 16, 8, ((700, 5000), (701, 3))),      # a long cache among them: an item that is cut
    (3000, (0, 2), 30, 8, 4, ((2999, 2000),)),               # several refills, sequences without tokens
    (700, (1, 30), 60, 16, 8, ()),                           # a few tokens each
])
def test_tokens(gdn_lib, n, q, k, Hq, Hk, long):
    ql, kl = lengths(n, q, k, seed=n, long=long)
    assert most_items(ql, kl, Hq // Hk, Hk, True) > constant("BATCH")
    x = paged.cache(ql, kl, Hq, Hk, 16, seed=n)
    both(gdn_lib, x, ql, kl, most=max(kl), weights=n == 700)


@pytest.mark.parametrize("n,q,k,Hq,Hk,long", [
    (500, (0, 90), 50, 8, 8, ()),                            # an item to a sequence, one query tile
    (400, (100, 220), 50, 8, 8, ()),                         # two query tiles of 128 tokens
    (700, (0, 70), 30, 16, 4, ((150, 4000), (151, 9000))),   # several items to a sequence, some cut
    (1500, (1, 40), 20, 16, 1, ()),                          # 8 tokens to a tile, pairs of tiles and single ones
    (3000, (0, 3), 12, 8, 4, ((5, 3000),)),
])
def test_prompts(gdn_lib, n, q, k, Hq, Hk, long):
    ql, kl = lengths(n, q, k, seed=n, long=long)
    ql[n // 3], kl[n // 3] = 300, 310       # (longer than a query tile: the kernel for many rows)
    assert most_items(ql, kl, Hq // Hk, Hk, False) > constant("BATCH")
    x = paged.cache(ql, kl, Hq, Hk, 16, seed=n)
    both(gdn_lib, x, ql, kl, most=max(kl), weights=n == 700)


def test_repeated_and_in_a_graph(gdn_lib):
    """The same bits each time, and from a graph."""
    for ql, kl in (lengths(1500, (1, 1), 20, seed=1, long=((700, 5000),)), lengths(400, (0, 220), 50, seed=2)):
        d = paged.cuda(paged.cache(ql, kl, 8, 8, 16, seed=3))
        call = lambda: gdn_lib.attn_paged(d["q"], d["kp"], d["vp"], d["table"], d["k_len"], cu_q=d["cu"], max_q=max(ql))
        first, again = call(), call()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            got = call()
        graph.replay()
        torch.cuda.synchronize()
        for other in (again, got):
            assert all(torch.equal(a, b) for a, b in zip(first, other))
