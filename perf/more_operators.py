"""The operators around a softmax layer that is served from a paged cache, as measured cases.

Norms of query and key heads with the position rotation in the same pass (with its gradients, and the form that
writes new keys and values into a cache's pages), attention of new tokens over the pages, the attention weight
that each cached key has received, and the eviction of the lightest keys.  A case is one pass through one operator.
With `own` false, `run` computes it in elementary torch operations in 32 bits; with `own` true it calls this
framework's operators.  `exact` gives the same outputs in 64 bits, from the definitions.

Formulas, per token t and head, with heads of 128 values of which the first 2 P are rotated:
  rope:     n = x rsqrt(mean(x^2) + eps) w,  y = n with each pair (a, b) turned by pos[axis_j, t] f_j, j < P
  attend:   o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys j <= i + (keys - queries) of the sequence,
            whose row j lies in page table[j // page] at j % page
  weigh:    weight_j += sum over queries i and heads h of the key head's group of exp(scale q_ih . k_j - lse_ih)
  evict:    the last `recent` keys of a sequence stay, and of the others the heaviest, `budget` in all; they move
            in their order to the first rows of the pages that `to` lists
"""
import math

import torch

own = False

D = 128      # head size
EPS = 1e-6


# ---- cases ----------------------------------------------------------------------------------------------

def listed():
    return [
        # a short prompt's heads: latency counts
        {"name": "rope_prompt_77", "op": "rope", "train": False, "n": 77, "Hq": 16, "Hk": 4, "norm": True, "axes": "1",
         "pairs": 64, "interleaved": False, "far": 0},
        # a training step's pass over packed documents: forward, then the gradients, those of the norms' weights among them
        {"name": "rope_train_8192", "op": "rope", "train": True, "n": 8192, "Hq": 16, "Hk": 4, "norm": True, "axes": "1",
         "pairs": 64, "interleaved": False, "far": 0},
        # the same for the patches of a clip of 9 frames of 30 x 52, heads without groups
        {"name": "rope_train_clip", "op": "rope", "train": True, "n": 14040, "Hq": 16, "Hk": 16, "norm": True,
         "axes": "16,24,24", "pairs": 64, "interleaved": False, "far": 0},
        # the next token of 64 users far into their contexts, keys and values into the cache's pages
        {"name": "rope_append_64", "op": "append", "n": 64, "Hq": 16, "Hk": 4, "norm": True, "axes": "1", "pairs": 64,
         "interleaved": False, "far": 1000000, "page": 64},
        # one user's next token over a short context: latency counts
        {"name": "attend_token_1", "op": "attend", "q": "1", "k": "777", "page": 16, "Hq": 16, "Hk": 4},
        # the next token of 32 users whose contexts differ
        {"name": "attend_token_32", "op": "attend", "q": ",".join(["1"] * 32),
         "k": ",".join(str(1 + 523 * i) for i in range(32)), "page": 64, "Hq": 16, "Hk": 4},
        # a serving step: parts of three prompts beside the next tokens of 20 users, small pages
        {"name": "attend_mixed", "op": "attend", "q": "512,300,129," + ",".join(["1"] * 20),
         "k": "4096,300,9000," + ",".join(str(100 + 397 * i) for i in range(20)), "page": 16, "Hq": 16, "Hk": 2},
        # the last part of a long prompt
        {"name": "attend_chunk_2048", "op": "attend", "q": "2048", "k": "32768", "page": 128, "Hq": 16, "Hk": 4},
        # the weight that the next token of 32 users gives to what is cached
        {"name": "weigh_token_32", "op": "weigh", "q": ",".join(["1"] * 32),
         "k": ",".join(str(1 + 523 * i) for i in range(32)), "page": 64, "Hq": 16, "Hk": 4},
        # the weight that a long prompt and two short ones give to their own keys
        {"name": "weigh_prompts", "op": "weigh", "q": "8192,640,77", "k": "8192,640,77", "page": 64, "Hq": 16, "Hk": 4},
        # one user's cache halved
        {"name": "evict_1", "op": "evict", "k": "1024", "page": 16, "Hk": 4, "budget": 512, "recent": 128},
        # a full serving batch's caches down to a budget
        {"name": "evict_32", "op": "evict", "k": ",".join(str(1 + 523 * i) for i in range(32)), "page": 64, "Hk": 4,
         "budget": 4096, "recent": 1024},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _text(v):
    return ",".join(str(x) for x in v)


def _draw(rng):
    op = rng.choice(["rope", "rope", "append", "attend", "attend", "weigh", "weigh", "evict"])
    Hk = rng.choice([1, 2, 4, 8, 16])
    page = rng.choice([16, 16, 32, 48, 64, 128, 256])
    if op in ("rope", "append"):
        pairs = rng.choice([64, 64, 64, 32, 16, 48])
        axes = rng.choice(["1", "1", "3", "2"]) if pairs != 64 else rng.choice(["1", "1", "3", "2", "16,24,24", "32,32"])
        c = {"op": op, "n": _log_int(rng, 1, 14040), "Hq": Hk * rng.choice([1, 2, 3, 4, 8]), "Hk": Hk, "norm": rng.random() < 0.7,
             "axes": axes, "pairs": pairs, "interleaved": rng.random() < 0.4, "far": rng.choice([0, 0, 30000, 1000000])}
        if op == "append":
            c["page"] = page
        else:
            c["train"] = rng.random() < 0.6
        return c
    if op == "evict":
        n, most = _log_int(rng, 1, 32), _log_int(rng, 64, 16384)
        budget = _log_int(rng, 16, most)
        return {"op": op, "k": _text(rng.randint(0, most) for _ in range(n)), "page": page, "Hk": Hk, "budget": budget,
                "recent": rng.choice([0, 1, budget // 4, budget // 2, budget])}
    Hk = min(Hk, 8)
    Hq = Hk * rng.choice([1, 2, 3, 4, 8])
    if rng.random() < 0.5:   # tokens, or a few each, of many users
        rows, most, few = _log_int(rng, 1, 64), _log_int(rng, 64, 16384), rng.choice([1, 1, 1, 4, 9])
        q = [rng.randint(1, few) for _ in range(rows)]
        k = [rng.randint(min(x, most), most) for x in q]
    else:                    # parts of prompts
        q = [_log_int(rng, 1, 4096) for _ in range(rng.choice([1, 1, 2, 3, 6]))]
        k = [x + rng.choice([0, 0, _log_int(rng, 1, 16384)]) for x in q]
    return {"op": op, "q": _text(q), "k": _text(k), "page": page, "Hq": Hq, "Hk": Hk}


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = [max(a, b) for a, b in zip(most.get(c["op"], (0, 0)), (w["bytes"], w["flops"]))]
    most["append"] = [max(most["append"][0], most["rope"][0] // 2), most["rope"][1]]
    while True:
        c = _draw(rng)
        w, top = work(c), most[c["op"]]
        if w["bytes"] <= top[0] and w["flops"] <= top[1]:
            return c


def _ints(text):
    return [int(x) for x in text.split(",")]


def work(case):
    op = case["op"]
    if op in ("rope", "append"):
        n, Hq, Hk = case["n"], case["Hq"], case["Hk"]
        A = len(_axes(case)[1])
        row = n * (Hq + Hk)
        if op == "append":  # k and v into the pages
            return {"bytes": 2 * (row + n * Hk) * 2 * D + 4 * n * (A + 1), "flops": 8 * D * row}
        return {"bytes": (4 if case["train"] else 2) * row * 2 * D + 4 * n * A, "flops": (24 if case["train"] else 8) * D * row}
    kl, Hk, page = _ints(case["k"]), case["Hk"], case["page"]
    tables = 4 * sum(-(-m // page) for m in kl)
    if op == "evict":
        kept = sum(min(m, case["budget"]) for m in kl)
        return {"bytes": 4 * Hk * sum(kl) + kept * Hk * (8 * D + 4) + 2 * tables, "flops": Hk * sum(kl)}
    ql, Hq = _ints(case["q"]), case["Hq"]
    pairs = sum(_pairs(a, b) for a, b in zip(ql, kl))
    nq, nk = sum(ql), sum(kl)
    if op == "weigh":
        return {"bytes": nq * Hq * (2 * D + 4) + nk * Hk * (2 * D + 8) + tables, "flops": 2 * D * pairs * Hq}
    return {"bytes": nq * Hq * (4 * D + 4) + nk * Hk * 4 * D + tables, "flops": 4 * D * pairs * Hq}


def _pairs(q, k):
    """(query, key) pairs that the causal mask leaves: query i sees keys j <= i + k - q."""
    first = max(0, q - k)          # rows before this one see nothing
    n = q - first
    return n * (k - q + first + 1) + n * (n - 1) // 2 if n > 0 else 0


def _axes(case):
    """(axis of each pair, the axes): "2" or "3" takes the axes in turn, "16,24,24" one behind another."""
    P, text = case["pairs"], case["axes"]
    if "," in text:
        parts = _ints(text)
        return [a for a, m in enumerate(parts) for _ in range(m)], range(len(parts))
    return [j % int(text) for j in range(P)], range(int(text))


# ---- inputs ---------------------------------------------------------------------------------------------

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    bf = torch.bfloat16

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32).to(dev)

    def perm(n):
        return torch.randperm(n, generator=gen, device=dev).to(torch.int32)

    s = dict(case)
    op = case["op"]
    if op in ("rope", "append"):
        n, Hq, Hk, P = case["n"], case["Hq"], case["Hk"], case["pairs"]
        axis, axes = _axes(case)
        s["axis"] = tuple(axis) if len(axes) > 1 else None
        s["freq"] = torch.exp2(-torch.arange(P, device=dev, dtype=torch.float64) * math.log2(1e6) / P).float()
        # the projection's rows, of which q, k and v are parts
        s["qkv"] = (normal(n, (Hq + 2 * Hk) * D) * 1.5).to(bf)
        s["wq"], s["wk"] = (normal(2, D) * 0.1 + 1.0).unbind(0) if case["norm"] else (None, None)
        t = torch.arange(n, device=dev, dtype=torch.int32)
        if len(axes) > 1:        # frames, lines and columns of patches
            side = max(1, int(math.sqrt(n / 9)))
            grid = [t // (side * side), t // side % side, t % side]
            s["pos"] = torch.stack([grid[a] + case["far"] for a in axes])
        elif op == "append":     # each token at the end of its own context
            s["pos"] = (torch.rand(n, generator=gen, device=dev) * (case["far"] + 100)).to(torch.int32)
        else:                    # documents one behind another
            s["pos"] = t % max(1, (n + 3) // 4) + case["far"]
        if op == "append":
            pages = n // case["page"] + 5
            s["kp"], s["vp"] = normal(pages, case["page"], Hk, D).to(bf), normal(pages, case["page"], Hk, D).to(bf)
            s["slots"] = perm(pages * case["page"])[:n]
            if n > 8:
                s["slots"][n // 2] = -1    # a padded row of the batch
        elif case["train"]:
            s["gq"], s["gk"] = normal(n, Hq, D).to(bf), normal(n, Hk, D).to(bf)
        return s
    kl, page, Hk = _ints(case["k"]), case["page"], case["Hk"]
    most = max(1, max(-(-m // page) for m in kl))
    kept = [-(-min(m, case["budget"]) // page) for m in kl] if op == "evict" else [0] * len(kl)
    total = sum(-(-m // page) for m in kl) + sum(kept) + 3
    order = perm(total)
    s["len"] = ints(kl)

    def table(counts, at):   # each sequence's pages, -1 behind them
        rows = torch.full((len(kl), most), -1, dtype=torch.int32, device=dev)
        for b, m in enumerate(counts):
            rows[b, :m] = order[at:at + m]
            at += m
        return rows

    s["table"] = table([-(-m // page) for m in kl], 0)
    s["kp"] = normal(total, page, Hk, D).to(bf)
    if op == "evict":
        s["vp"] = normal(total, page, Hk, D).to(bf)
        s["to"] = table(kept, sum(-(-m // page) for m in kl))
        s["weights"] = torch.exp(2.0 * normal(total, Hk, page))
        return s
    ql, Hq = _ints(case["q"]), case["Hq"]
    s["cu"] = ints([0] + ql).cumsum(0).to(torch.int32)
    s["max_q"], s["max_k"] = max(ql), max(kl)
    s["tq"] = normal(sum(ql), Hq, D).to(bf)
    if op == "attend":
        s["vp"] = normal(total, page, Hk, D).to(bf)
    else:
        s["weights"] = torch.exp(normal(total, Hk, page))
        s["lse"] = torch.cat([_scores(s, b, ql, kl)[0].logsumexp(-1).permute(2, 0, 1).reshape(ql[b], Hq)
                              for b in range(len(ql)) if ql[b]])
    return s


# ---- one pass -------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "weigh": _plain_weigh,
            "evict": _plain_evict}[s["op"]](s)


def _split(s):
    """q, k, v as parts of the projection's rows."""
    return [x.unflatten(1, (-1, D)) for x in s["qkv"].split([s["Hq"] * D, s["Hk"] * D, s["Hk"] * D], 1)]


def _run_own(s):
    import linear_attention_rnn_gb300 as gdn

    op = s["op"]
    if op in ("rope", "append"):
        q, k, v = _split(s)
        how = dict(q_weight=s["wq"], k_weight=s["wk"], eps=EPS, pair_axis=s["axis"], interleaved=s["interleaved"])
        if op == "append":
            qo = gdn.rope_append(q, k, v, s["pos"], s["freq"], s["kp"], s["vp"], s["slots"], **how)
            return {"q": qo, "k_pages": s["kp"], "v_pages": s["vp"]}
        qo, ko = gdn.rope_fwd(q, k, s["pos"], s["freq"], **how)
        if not s["train"]:
            return {"q": qo, "k": ko}
        dq, dk, dwq, dwk = gdn.rope_bwd(q, k, s["pos"], s["freq"], s["gq"], s["gk"], **how)
        return _without_none({"q": qo, "k": ko, "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk})
    if op == "evict":
        n = gdn.cache_evict(s["kp"], s["vp"], s["weights"], s["table"], s["len"], s["budget"], recent=s["recent"],
                            to_table=s["to"])
        return {"len": n, "k_pages": s["kp"], "v_pages": s["vp"], "weights": s["weights"]}
    at = dict(cu_q=s["cu"], max_q=s["max_q"], max_k=s["max_k"])
    if op == "weigh":
        return {"weights": gdn.attn_paged_weights(s["tq"], s["kp"], s["lse"], s["table"], s["len"], s["weights"], **at)}
    o, lse = gdn.attn_paged(s["tq"], s["kp"], s["vp"], s["table"], s["len"], **at)
    return {"o": o, "lse": lse}


def _without_none(d):
    return {k: v for k, v in d.items() if v is not None}


def _turns(s):
    """cos and sin of every token's angles, [n, 1, P]; the angles in 64 bits, which far positions need."""
    pos = s["pos"] if s["pos"].dim() == 2 else s["pos"][None]
    axis = torch.tensor(s["axis"] or [0] * s["pairs"], device=pos.device)
    angle = (pos[axis].T.double() * s["freq"].double())[:, None]
    return angle.cos().float(), angle.sin().float()


def _turn(x, cos, sin, s):
    """The pairs of the first 2 P values turned."""
    P = s["pairs"]
    r, rest = x[..., :2 * P], x[..., 2 * P:]
    if s["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :P], r[..., P:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _unit(x, w):
    """(x over its root mean square, the factor): x itself without a weight."""
    if w is None:
        return x, None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _plain_heads(x, w, cos, sin, s):
    u, _ = _unit(x.float(), w)
    return _turn(u if w is None else u * w, cos, sin, s).to(x.dtype)


def _plain_heads_bwd(x, w, dy, cos, sin, s):
    dn = _turn(dy.float(), cos, -sin, s)
    if w is None:
        return dn.to(x.dtype), None
    u, r = _unit(x.float(), w)
    g = dn * w
    dx = r * (g - u * (g * u).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dn * u).sum((0, 1), dtype=torch.float64).float()


def _plain_rope(s):
    q, k, _ = _split(s)
    cos, sin = _turns(s)
    out = {"q": _plain_heads(q, s["wq"], cos, sin, s), "k": _plain_heads(k, s["wk"], cos, sin, s)}
    if s["train"]:
        out["dq"], dwq = _plain_heads_bwd(q, s["wq"], s["gq"], cos, sin, s)
        out["dk"], dwk = _plain_heads_bwd(k, s["wk"], s["gk"], cos, sin, s)
        out.update({"dwq": dwq, "dwk": dwk})
    return _without_none(out)


def _plain_append(s):
    q, k, v = _split(s)
    cos, sin = _turns(s)
    k = _plain_heads(k, s["wk"], cos, sin, s)
    to = torch.where(s["slots"] < 0, s["kp"].shape[0] * s["page"], s["slots"].long())
    for pages, rows in ((s["kp"], k), (s["vp"], v)):
        flat = pages.view(-1, *pages.shape[2:])
        at = (to < flat.shape[0]).nonzero()[:, 0]
        flat[to[at]] = rows[at]
    return {"q": _plain_heads(q, s["wq"], cos, sin, s), "k_pages": s["kp"], "v_pages": s["vp"]}


def _rows(s, b, m):
    """(page, row in it) of the first m keys of sequence b."""
    j = torch.arange(m, device=s["table"].device)
    return s["table"][b, j // s["page"]].long(), j % s["page"]


def _scores(s, b, ql, kl):
    """Scaled scores of sequence b, [Hk, G, queries, keys], minus infinity where masked; and the keys' places."""
    n, m, at = ql[b], kl[b], sum(ql[:b])
    page, row = _rows(s, b, m)
    K = s["kp"][page, row].float().permute(1, 2, 0)[:, None]                        # [Hk, 1, D, m]
    Q = s["tq"][at:at + n].float().unflatten(1, (s["Hk"], -1)).permute(1, 2, 0, 3)  # [Hk, G, n, D]
    z = (Q @ K).mul_(D ** -0.5)
    i, j = torch.arange(n, device=z.device), torch.arange(m, device=z.device)
    return z.masked_fill_(j[None] > i[:, None] + (m - n), -math.inf), page, row


def _plain_attend(s):
    ql, kl = _ints(s["q"]), _ints(s["k"])
    o, lse = [], []
    for b in range(len(ql)):
        z, page, row = _scores(s, b, ql, kl)
        if kl[b] == 0:
            o.append(torch.zeros(ql[b], s["Hq"], D, dtype=s["tq"].dtype, device=z.device))
            lse.append(torch.full((ql[b], s["Hq"]), -math.inf, device=z.device))
            continue
        top = z.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        p = z.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        V = s["vp"][page, row].float().permute(1, 0, 2)[:, None]
        y = (p @ V) / torch.where(total == 0, 1.0, total)
        o.append(y.permute(2, 0, 1, 3).flatten(1, 2).to(s["tq"].dtype))
        lse.append((top + torch.log(total))[..., 0].permute(2, 0, 1).flatten(1, 2))
    return {"o": torch.cat(o), "lse": torch.cat(lse)}


def _plain_weigh(s):
    ql, kl = _ints(s["q"]), _ints(s["k"])
    at = 0
    for b in range(len(ql)):
        z, page, row = _scores(s, b, ql, kl)
        l = s["lse"][at:at + ql[b]].unflatten(1, (s["Hk"], -1)).permute(1, 2, 0)[..., None]
        at += ql[b]
        p = torch.where(z == -math.inf, 0.0, z.sub_(l).exp_())
        s["weights"][page, :, row] += p.sum((1, 2)).T
    return {"weights": s["weights"]}


def _plain_evict(s):
    kl, budget = _ints(s["k"]), s["budget"]
    new = []
    for b, m in enumerate(kl):
        recent = min(s["recent"], budget, m)
        old = m - recent
        take = min(budget - recent, old)
        page, row = _rows(s, b, m)
        w = s["weights"][page, :, row].T                                             # [Hk, m]
        first = torch.sort(w[:, :old], dim=1, descending=True, stable=True).indices[:, :take].sort(1).values
        last = torch.arange(old, m, device=w.device).expand(s["Hk"], -1)
        keep = torch.cat([first, last], 1)                                           # [Hk, kept]
        j = torch.arange(keep.shape[1], device=w.device)
        to, place = s["to"][b, j // s["page"]].long(), j % s["page"]
        h = torch.arange(s["Hk"], device=w.device)[:, None]
        for pages in (s["kp"], s["vp"]):
            pages[to, place, h] = pages[page[keep], row[keep], h]
        s["weights"][to, h, place] = w.gather(1, keep)
        new.append(keep.shape[1])
    return {"len": torch.tensor(new, dtype=torch.int32, device="cuda"), "k_pages": s["kp"], "v_pages": s["vp"],
            "weights": s["weights"]}


# ---- the definitions in 64 bits -------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_rope, "attend": _exact_attention, "weigh": _exact_attention,
            "evict": _exact_evict}[case["op"]](s, case)


def _exact_rope(s, case):
    """Head by head, each pair as a complex number times e^(i angle)."""
    n, Hq, Hk, P = case["n"], case["Hq"], case["Hk"], case["pairs"]
    x = s["qkv"].double().view(n, Hq + 2 * Hk, D)
    pos = s["pos"].double().reshape(-1, n)
    axis, _ = _axes(case)
    angle = torch.stack([pos[a] * s["freq"][j].double() for j, a in enumerate(axis)], 1)
    e = torch.polar(torch.ones_like(angle), angle)
    first = torch.arange(P, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else P)

    def turned(y, e):
        z = torch.complex(y[:, first], y[:, second]) * e
        y = y.clone()
        y[:, first], y[:, second] = z.real, z.imag
        return y

    def scale(y):
        return 1.0 / torch.sqrt(y.square().sum(1) / D + EPS)

    def forward(h, w):
        y = x[:, h]
        return turned(y if w is None else y * scale(y)[:, None] * w.double(), e)

    q = torch.stack([forward(h, s["wq"]) for h in range(Hq)], 1)
    k = torch.stack([forward(Hq + h, s["wk"]) for h in range(Hk)], 1)
    if case["op"] == "append":
        kp, vp = s["kp"].double(), s["vp"].double()
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                kp[slot // case["page"], slot % case["page"]] = k[t]
                vp[slot // case["page"], slot % case["page"]] = x[t, Hq + Hk:]
        return {"q": q, "k_pages": kp, "v_pages": vp}
    if not case["train"]:
        return {"q": q, "k": k}

    def backward(h, w, dy):
        dn = turned(dy.double(), e.conj())
        if w is None:
            return dn, None
        y, r = x[:, h], scale(x[:, h])
        # y_j r: d(y_j r) / dy_i = r delta_ij - r^3 y_i y_j / D
        g = dn * w.double()
        dx = r[:, None] * g - (r ** 3 * (g * y).sum(1) / D)[:, None] * y
        return dx, (dn * y * r[:, None]).sum(0)

    out = {"q": q, "k": k}
    for name, heads, base, w, dy in (("q", Hq, 0, s["wq"], s["gq"]), ("k", Hk, Hq, s["wk"], s["gk"])):
        parts = [backward(base + h, w, dy[:, h]) for h in range(heads)]
        out["d" + name] = torch.stack([p[0] for p in parts], 1)
        if w is not None:
            out["dw" + name] = sum(p[1] for p in parts)
    return {key: out[key] for key in ("q", "k", "dq", "dk", "dwq", "dwk") if key in out}


def _exact_attention(s, case):
    """Sequence by sequence and head by head, the keys gathered row by row from their pages."""
    ql, kl, Hq, Hk, page = _ints(case["q"]), _ints(case["k"]), case["Hq"], case["Hk"], case["page"]
    weigh = case["op"] == "weigh"
    if sum(a * b for a, b in zip(ql, kl)) * Hq > 2e9:   # (the widest products: some ten seconds)
        return None
    table, start = s["table"].tolist(), s["cu"].tolist()
    w = s["weights"].double() if weigh else None
    o = torch.zeros(sum(ql), Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(ql), Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, m) in enumerate(zip(ql, kl)):
        if n == 0 or m == 0:
            continue
        flat = torch.tensor([table[b][j // page] * page + j % page for j in range(m)], device="cuda")
        hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1)
        rows = slice(start[b], start[b] + n)
        for h in range(Hq):
            kh = h // (Hq // Hk)
            K = s["kp"].view(-1, Hk, D)[flat, kh].double()
            z = (s["tq"][rows, h].double() @ K.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
            if weigh:
                w[flat // page, kh, flat % page] += torch.exp(z - s["lse"][rows, h].double()[:, None]).sum(0)
                continue
            l = torch.logsumexp(z, 1)
            lse[rows, h] = l
            p = torch.exp(z - torch.where(l == -math.inf, 0.0, l)[:, None])
            o[rows, h] = p @ s["vp"].view(-1, Hk, D)[flat, kh].double()
    return {"weights": w} if weigh else {"o": o, "lse": lse}


def _exact_evict(s, case):
    """A key stays when fewer than `take` others weigh more, or as much at a lower index."""
    page, Hk, budget = case["page"], case["Hk"], case["budget"]
    table, to = s["table"].tolist(), s["to"].tolist()
    kp, vp, w = s["kp"].double(), s["vp"].double(), s["weights"].double()
    new = []
    for b, m in enumerate(_ints(case["k"])):
        recent = min(case["recent"], budget, m)
        take = min(budget - recent, m - recent)
        src = torch.tensor([table[b][j // page] * page + j % page for j in range(m)], device="cuda", dtype=torch.long)
        for h in range(Hk):
            x = w[:, h].reshape(-1)[src[:m - recent]]
            order = sorted(range(m - recent), key=x.tolist().__getitem__, reverse=True)[:take]  # (keeps ties in order)
            keep = torch.tensor(sorted(order) + list(range(m - recent, m)), device="cuda", dtype=torch.long)
            dst = torch.tensor([to[b][i // page] * page + i % page for i in range(len(keep))], device="cuda", dtype=torch.long)
            for pages, source in ((kp, s["kp"]), (vp, s["vp"])):
                pages.view(-1, Hk, D)[dst, h] = source.view(-1, Hk, D)[src[keep], h].double()
            w[dst // page, h, dst % page] = s["weights"][src[keep] // page, h, src[keep] % page].double()
        new.append(min(m, budget))
    return {"len": torch.tensor(new, dtype=torch.int32, device="cuda"), "k_pages": kp, "v_pages": vp, "weights": w}
