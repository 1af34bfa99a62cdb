"""Softmax attention layers served from a paged cache: prompts read by chunks beside single
tokens of other sequences, pages handed out as sequences grow, and the lightest keys evicted
where a cache has reached its budget.

    python examples/paged_serving.py

Each layer norms its query and key heads and turns them by their positions (rope_append, which
also writes keys and values into the pages), attends over the pages (attn_paged) and adds
up the weight that each key receives (attn_paged_weights); cache_evict keeps the
heaviest and the latest keys.  Weights are random.  Without eviction the outputs are those of one
pass over whole prompts (rope_fwd and attn_fwd), which main() compares.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_rnn_gb300 as gdn  # noqa: E402

D = 128  # head size


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Cache:
    """The pages of one layer's keys and values, and the weight that each key has received."""

    def __init__(self, pages, page, Hk):
        self.k, self.v = (torch.empty(pages, page, Hk, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        self.weights = torch.zeros(pages, Hk, page, device="cuda")


class Sequences:
    """What the host keeps of the sequences: their pages, the keys in them, their next position."""

    def __init__(self, pages, page, most):
        self.page, self.most = page, most     # rows of a page, pages of a sequence
        self.free = list(range(pages))
        self.pages, self.keys, self.position = {}, {}, {}

    def grow(self, name, n):
        """Room for n more keys; their places in the cache and their positions."""
        pages, k, p = self.pages.setdefault(name, []), self.keys.get(name, 0), self.position.get(name, 0)
        while len(pages) * self.page < k + n:
            pages.append(self.free.pop())
        self.keys[name], self.position[name] = k + n, p + n
        return [pages[j // self.page] * self.page + j % self.page for j in range(k, k + n)], list(range(p, p + n))

    def table(self, names):
        return ints([self.pages[s] + [-1] * (self.most - len(self.pages[s])) for s in names])

    def shrink(self, name, keys):
        self.keys[name] = keys
        while len(self.pages[name]) * self.page >= keys + self.page:
            self.free.append(self.pages[name].pop())


class Layer:
    def __init__(self, width, Hq, Hk, gen):
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        self.parts = [Hq * D, Hk * D, Hk * D]
        self.w = (r(width, sum(self.parts)) * width ** -0.5).bfloat16()
        self.out = (r(Hq * D, width) * (Hq * D) ** -0.5).bfloat16()
        self.q_weight, self.k_weight = (1 + 0.1 * r(D) for _ in "qk")

    def split(self, x):
        return [t.unflatten(-1, (-1, D)) for t in (x @ self.w).split(self.parts, -1)]

    def norms(self):
        return dict(q_weight=self.q_weight, k_weight=self.k_weight)


class Stack:
    def __init__(self, layers=2, width=512, Hq=8, Hk=2, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.width, self.Hk = width, Hk
        self.freq = torch.exp2(-torch.arange(D // 2, dtype=torch.float64) * 20 / (D // 2)).float().cuda()
        self.layers = [Layer(width, Hq, Hk, gen) for _ in range(layers)]

    def whole(self, x, lens):
        """One pass over packed prompts, without a cache."""
        cu = ints([0] + lens).cumsum(0).to(torch.int32)
        pos = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in lens])
        for m in self.layers:
            q, k, v = m.split(x)
            q, k = gdn.rope_fwd(q, k, pos, self.freq, **m.norms())
            o, _ = gdn.attn_fwd(q, k, v, cu_q=cu, cu_k=cu, max_q=max(lens), max_k=max(lens))
            x = x + o.flatten(-2) @ m.out
        return x

    def step(self, parts, seqs, caches):
        """One serving step: `parts` lists (sequence, its new rows).  Returns the new rows' outputs."""
        names, lens = [s for s, _ in parts], [t.shape[0] for _, t in parts]
        grown = [seqs.grow(s, n) for s, n in zip(names, lens)]
        slots, pos = (ints([x for g in grown for x in g[i]]) for i in range(2))
        table, k_len = seqs.table(names), ints([seqs.keys[s] for s in names])
        at = dict(cu_q=ints([0] + lens).cumsum(0).to(torch.int32), max_q=max(lens), max_k=max(seqs.keys[s] for s in names))
        x = torch.cat([t for _, t in parts])
        for m, c in zip(self.layers, caches):
            q, k, v = m.split(x)
            q = gdn.rope_append(q, k, v, pos, self.freq, c.k, c.v, slots, **m.norms())
            o, lse = gdn.attn_paged(q, c.k, c.v, table, k_len, **at)
            gdn.attn_paged_weights(q, c.k, lse, table, k_len, c.weights, **at)
            x = x + o.flatten(-2) @ m.out
        return x.split(lens)

    def evict(self, names, seqs, caches, budget, recent):
        """Every layer keeps its own keys; all of them as many."""
        table, k_len = seqs.table(names), ints([seqs.keys[s] for s in names])
        for c in caches:
            kept = gdn.cache_evict(c.k, c.v, c.weights, table, k_len, budget, recent=recent)
            at = torch.arange(table.shape[1] * seqs.page, device="cuda")  # rows behind them have no weight yet
            for b, n in enumerate(kept.tolist()):
                gone = at[(at >= n) & (at < int(k_len[b]))]
                c.weights[table[b, gone // seqs.page].long(), :, gone % seqs.page] = 0
        for s, n in zip(names, kept.tolist()):
            seqs.shrink(s, n)


def serve(lens=(300, 77), chunk=128, page=32, budget=None, recent=16, seed=1, **kw):
    """Prompts by chunks, each chunk beside the next tokens of the sequences that are through; the
    outputs of all rows.  With a budget, caches that exceed it are cut back after every step."""
    stack = Stack(**kw)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows = [torch.randn(n, stack.width, generator=gen, device="cuda").bfloat16() for n in lens]
    most = -(-max(lens) // page) + 1
    caches = [Cache(most * len(lens), page, stack.Hk) for _ in stack.layers]
    seqs, done, outs = Sequences(most * len(lens), page, most), [0] * len(lens), [[] for _ in lens]
    while any(d < n for d, n in zip(done, lens)):
        parts, left = [], chunk
        for s, (d, n) in enumerate(zip(done, lens)):
            # the second half of each prompt arrives token by token
            take = min(left, n // 2 - d) if d < n // 2 else min(1, n - d)
            if take > 0:
                parts.append((s, rows[s][d:d + take]))
                done[s], left = d + take, left - take
        for (s, _), o in zip(parts, stack.step(parts, seqs, caches)):
            outs[s].append(o)
        over = [s for s, _ in parts if budget is not None and seqs.keys[s] > budget]
        if over:
            stack.evict(over, seqs, caches, budget, recent)
    return stack, rows, [torch.cat(o) for o in outs], seqs


def main():
    gdn.lib()
    stack, rows, outs, _ = serve()
    ref = stack.whole(torch.cat(rows), [t.shape[0] for t in rows])
    diff = float((torch.cat(outs).float() - ref.float()).abs().max() / ref.float().abs().max())
    print(f"chunks and tokens over pages: largest difference from one pass {diff:.1e} of the largest output")
    _, _, outs, seqs = serve(budget=64)
    print("with a budget of 64 keys:", {s: n for s, n in seqs.keys.items()}, "keys left of", {s: n for s, n in seqs.position.items()})


if __name__ == "__main__":
    main()
