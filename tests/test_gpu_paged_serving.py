"""The operators of a paged cache together, as a serving loop runs them: prompts into pages by chunks,
tokens one by one, eviction when a cache is full; on a side stream and as captured graphs."""
import pytest
import torch

import paged
from oracle import ops
from test_gpu_attn import close

pytestmark = pytest.mark.gpu
Hq, Hk, PAGE = 4, 2, 32


def rows(n, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    return dict(q=r(n, Hq, 128).bfloat16(), k=r(n, Hk, 128).bfloat16(), v=r(n, Hk, 128).bfloat16())


W = dict(q_weight=1 + 0.1 * torch.arange(128) / 128, k_weight=1 - 0.1 * torch.arange(128) / 128)
FREQ = torch.exp2(-torch.arange(64, dtype=torch.float64) * 13 / 64).float()


def step(gdn, x, cache, table, k_len, cu, weights):
    """New tokens of every sequence: into the cache, over it, and their weights."""
    q = gdn.rope_append(x["q"], x["k"], x["v"], x["pos"], x["freq"], *cache, x["slots"], q_weight=x["wq"], k_weight=x["wk"])
    o, lse = gdn.attn_paged(q, *cache, table, k_len, cu_q=cu)
    gdn.attn_paged_weights(q, cache[0], lse, table, k_len, weights, cu_q=cu)
    return o, lse


def test_chunks_tokens_and_eviction(gdn_lib):
    """Two sequences read by chunks and token by token give what one pass over packed rows gives; after an
    eviction, what attention over the keys that stay gives.

    Tolerance: q and k are rounded to bf16 once by rope in either route (equal bits), so the attention's own
    bounds hold."""
    gdn, lens = gdn_lib, [150, 70]
    x = [rows(n, seed=n) for n in lens]
    wq, wk, freq = W["q_weight"].float().cuda(), W["k_weight"].float().cuda(), FREQ.cuda()
    P = 16
    cache = [torch.full((P, PAGE, Hk, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    weights = torch.zeros(P, Hk, PAGE, device="cuda")
    table = torch.tensor([[3, 9, 1, 7, 5], [2, 8, 0, -1, -1]], dtype=torch.int32)
    dt = table.cuda()
    done, outs = [0, 0], [[], []]
    for chunk in [(100, 1), (0, 40)] + [(1, 1)] * 29 + [(21, 0)]:
        part = {n: torch.cat([x[s][n][done[s]:done[s] + c] for s, c in enumerate(chunk)]).cuda() for n in "qkv"}
        pos = [p for s, c in enumerate(chunk) for p in range(done[s], done[s] + c)]
        slots = [int(table[s, p // PAGE]) * PAGE + p % PAGE for s, c in enumerate(chunk) for p in range(done[s], done[s] + c)]
        part.update(pos=paged.ints(pos).cuda(), slots=paged.ints(slots).cuda(), freq=freq, wq=wq, wk=wk)
        done = [d + c for d, c in zip(done, chunk)]
        o, _ = step(gdn, part, cache, dt, paged.ints(done).cuda(), paged.cu(chunk).cuda(), weights)
        for s, t in enumerate(o.split(list(chunk))):
            outs[s].append(t)
    assert done == lens
    cu = paged.cu(lens).cuda()
    whole = {n: torch.cat([y[n] for y in x]).cuda() for n in "qkv"}
    pos = paged.ints(list(range(150)) + list(range(70))).cuda()
    q, k = gdn.rope_fwd(whole["q"], whole["k"], pos, freq, q_weight=wq, k_weight=wk)
    kl0 = [0, 150]
    eps = float(128 ** -0.5 * q.float().norm(dim=-1).max() * k.float().norm(dim=-1).max() * 136 * 2.0 ** -23)
    r = ops.attn(q, k, whole["v"], lens, kl0, lens, 128 ** -0.5, eps=eps)
    close(torch.cat([torch.cat(t) for t in outs]), r["o"], r["o_tol"], "o by chunks and tokens")
    # every query spreads a weight of one for each head, over the keys in all
    total = torch.stack([sum(weights[int(e), :, :min(PAGE, n - PAGE * i)].sum(1) for i, e in enumerate(table[s]) if e >= 0 and n > PAGE * i)
                         for s, n in enumerate(lens)])
    assert torch.allclose(total.cpu(), torch.tensor([[150.0 * Hq / Hk] * Hk, [70.0 * Hq / Hk] * Hk]), rtol=1e-4)
    # down to 64 keys each, 16 of them the last ones, in place
    host = [t.cpu() for t in cache] + [weights.cpu()]
    want = ops.cache_evict(*host, table, lens, 64, 16, table)
    n = gdn.cache_evict(*cache, weights, dt, paged.ints(lens).cuda(), 64, recent=16)
    assert n.tolist() == [64, 64] == want[3]
    # the next tokens: over what stayed, their own keys behind it
    new = {k: torch.cat([rows(1, seed=50 + s)[k] for s in range(2)]).cuda() for k in "qkv"}
    new.update(pos=paged.ints(lens).cuda(), slots=paged.ints([int(table[s, 64 // PAGE]) * PAGE for s in range(2)]).cuda(),
               freq=freq, wq=wq, wk=wk)
    o, lse = step(gdn, new, cache, dt, n + 1, paged.cu([1, 1]).cuda(), weights)
    q, k = gdn.rope_fwd(new["q"], new["k"], new["pos"], freq, q_weight=wq, k_weight=wk)
    for s in range(2):
        want[0][table[s, 2], 0], want[1][table[s, 2], 0] = k[s].cpu(), new["v"][s].cpu()
    r = ops.attn_paged(q, want[0], want[1], table, [1, 1], [65, 65], 128 ** -0.5, eps)
    close(o, r["o"], r["o_tol"], "o after the eviction")


def inputs(seed, ql, kl):
    x = paged.cuda(paged.cache(ql, kl, Hq, Hk, PAGE, seed=seed, spare=9, nan=False))
    r = {n: t.cuda() for n, t in rows(sum(ql), seed).items()}
    free = sorted(set(range(x["kp"].shape[0])) - set(x["table"].flatten().tolist()))
    slots = [int(x["table"][s, p // PAGE]) * PAGE + p % PAGE for s, (a, b) in enumerate(zip(ql, kl)) for p in range(b - a, b)]
    r.update(pos=paged.ints(range(sum(ql))).cuda() + 1000 * seed, slots=paged.ints(slots).cuda(), freq=FREQ.cuda(),
             wq=W["q_weight"].float().cuda(), wk=W["k_weight"].float().cuda(), kp=x["kp"], vp=x["vp"], table=x["table"],
             k_len=x["k_len"], cu=x["cu"], weights=x["weights"], gq=r["q"] * 0.5, gk=r["k"] * 0.5,
             to=torch.tensor(free[:8], dtype=torch.int32).view(2, 4).cuda())
    return r


def serve(gdn, x):
    """A serving step and a training pass of its heads: states in, outputs and states out."""
    cache, weights = [x["kp"].clone(), x["vp"].clone()], x["weights"].clone()
    o, lse = step(gdn, x, cache, x["table"], x["k_len"], x["cu"], weights)
    n = gdn.cache_evict(*cache, weights, x["table"], x["k_len"], 100, recent=30, to_table=x["to"])
    m = gdn.cache_evict(*cache, weights, x["table"], x["k_len"], 64, recent=3)
    back = gdn.rope_bwd(x["q"], x["k"], x["pos"], x["freq"], x["gq"], x["gk"], q_weight=x["wq"], k_weight=x["wk"])
    return (o, lse, *cache, weights, n, m, *back)


SHAPES = [([1, 1], [300, 77]), ([130, 20], [400, 20])]


@pytest.mark.parametrize("ql,kl", SHAPES)
def test_side_stream(gdn_lib, ql, kl):
    x = inputs(1, ql, kl)
    plain = serve(gdn_lib, x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = serve(gdn_lib, x)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, plain))


@pytest.mark.parametrize("ql,kl", SHAPES)
def test_captured_graph(gdn_lib, ql, kl):
    x = inputs(2, ql, kl)
    serve(gdn_lib, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = serve(gdn_lib, x)
    for seed in (3, 4):
        y = inputs(seed, ql, kl)
        for n in x:
            x[n].copy_(y[n])
        graph.replay()
        torch.cuda.synchronize()
        plain = serve(gdn_lib, y)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, plain))
