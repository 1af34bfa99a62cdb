"""The operators of a stack that alternates linear and softmax attention layers, as measured cases.

Linear attention with a decay for each head (a chunked form for prompts and training, a recurrent form for single
tokens), the gated delta rule's single-token form, and causal softmax attention with grouped heads over packed
sequences (prompts, training, single tokens over a cache).  A case is one pass through one operator.  With
`own` false, `run` computes it in elementary torch operations in 32 bits; with `own` true it calls this
framework's operators.  `exact` gives the same outputs in 64 bits, from the definitions.

Formulas, per sequence and (value) head, with token index t, log-decay w <= 0, and key head h // (Hv / Hk):
  decay:  S_t = e^w S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t,  S_{-1} = h0,  hT = S_{T-1}
  delta:  S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,  o_t = S_t^T q_t
  attn:   o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys j <= i + (keys - queries)
"""
import math

import torch

own = False

D = 128      # head size
CHUNK = 64   # tokens to a block of the plain chunked form


# ---- cases ----------------------------------------------------------------------------------------------

def listed():
    return [
        # a few short prompts (one of a single token, one empty) on a small model: latency counts
        {"name": "decay_prompt_short", "op": "decay", "train": False, "lens": "300,1,65,0", "Hk": 2, "Hv": 2, "h0": True},
        # one prompt of the layer benchmark's shape, continued from a state
        {"name": "decay_prompt_4096", "op": "decay", "train": False, "lens": "4096", "Hk": 16, "Hv": 32, "h0": True},
        # a long document read in one call
        {"name": "decay_prompt_65536", "op": "decay", "train": False, "lens": "65536", "Hk": 16, "Hv": 32, "h0": False},
        # a training step's pass over packed documents: forward, then the gradients
        {"name": "decay_train_packed", "op": "decay", "train": True, "lens": "4096,2500,1000,595,1", "Hk": 16, "Hv": 32,
         "h0": True},
        # one user's next token, and a full serving batch's
        {"name": "decay_step_1", "op": "decay_step", "rows": 1, "slots": 4, "Hk": 16, "Hv": 32},
        {"name": "decay_step_256", "op": "decay_step", "rows": 256, "slots": 300, "Hk": 16, "Hv": 32},
        # the same for the gated delta rule: a handful of users, and a large batch
        {"name": "delta_step_8", "op": "delta_step", "rows": 8, "slots": 8, "Hk": 16, "Hv": 32},
        {"name": "delta_step_512", "op": "delta_step", "rows": 512, "slots": 600, "Hk": 16, "Hv": 32},
        # prompts of mixed lengths packed into one call
        {"name": "attn_prompt_packed", "op": "attn", "train": False, "q": "3000,1,129,640,2048,77,1500,0,800", "k": "", "cap": 0,
         "Hq": 16, "Hk": 4},
        # one long prompt
        {"name": "attn_prompt_16384", "op": "attn", "train": False, "q": "16384", "k": "", "cap": 0, "Hq": 16, "Hk": 2},
        # a training step's pass over packed documents: forward, then the gradients
        {"name": "attn_train_packed", "op": "attn", "train": True, "q": "4096,2048,1000,977,71", "k": "", "cap": 0,
         "Hq": 16, "Hk": 4},
        # the next token of 32 users whose contexts differ, over caches of one capacity
        {"name": "attn_token_32", "op": "attn", "train": False, "q": ",".join(["1"] * 32),
         "k": ",".join(str(1 + 523 * i) for i in range(32)), "cap": 16384, "Hq": 16, "Hk": 4},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lens(rng, total):
    """Lengths that add up to `total`: one document, or some of different lengths, now and then an empty one."""
    n = rng.choice([1, 1, 2, 3, 5, 9, 17])
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _text(v):
    return ",".join(str(x) for x in v)


def _draw(rng):
    op = rng.choice(["decay", "decay", "decay_train", "decay_step", "delta_step", "attn", "attn_train", "attn_token"])
    Hk = rng.choice([1, 2, 4, 8, 16])
    if op.startswith("decay") and op != "decay_step":
        train = op == "decay_train"
        total = _log_int(rng, 64, 8192 if train else 65536)
        return {"op": "decay", "train": train, "lens": _text(_lens(rng, total)), "Hk": Hk, "Hv": Hk * rng.choice([1, 2, 4]),
                "h0": rng.random() < 0.5}
    if op.endswith("step"):
        rows = _log_int(rng, 1, 512)
        return {"op": op, "rows": rows, "slots": rows + rng.randint(0, 64), "Hk": Hk, "Hv": Hk * rng.choice([1, 2, 4])}
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4, 8])
    if op == "attn_token":
        rows, cap, most = _log_int(rng, 1, 64), _log_int(rng, 128, 16384), rng.choice([1, 1, 4, 9])
        q = [rng.randint(1, most) for _ in range(rows)]
        return {"op": "attn", "train": False, "q": _text(q), "k": _text(rng.randint(min(x, cap), cap) for x in q), "cap": cap,
                "Hq": Hq, "Hk": Hk}
    train = op == "attn_train"
    q = _lens(rng, _log_int(rng, 64, 8192 if train else 16384))
    # now and then a prompt that continues what is cached already (or, at its first rows, sees nothing)
    k = [x + rng.randint(-min(x, 40), 700) for x in q] if rng.random() < 0.3 else []
    return {"op": "attn", "train": train, "q": _text(q), "k": _text(k), "cap": 0, "Hq": Hq, "Hk": Hk}


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        at = (c["op"], c.get("train", False))
        most[at] = [max(a, b) for a, b in zip(most.get(at, (0, 0)), (w["bytes"], w["flops"]))]
    while True:
        c = _draw(rng)
        w, top = work(c), most[c["op"], c.get("train", False)]
        padded = max(_ints(c.get("q") or c.get("lens") or "1")) * len(_ints(c.get("q") or c.get("lens") or "1"))
        if w["bytes"] <= top[0] and w["flops"] <= top[1] and padded <= 65536:
            return c


def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _key_lens(case):
    return _ints(case["k"]) or _ints(case["q"])


def work(case):
    op = case["op"]
    if op == "decay":
        n, Hk, Hv = sum(_ints(case["lens"])), case["Hk"], case["Hv"]
        seqs = len(_ints(case["lens"]))
        state = seqs * Hv * D * D * 4
        rows = 2 * D
        b = n * (2 * Hk + 2 * Hv) * rows + state * (2 if case["h0"] else 1)
        f = 4 * D * D * n * Hv
        if case["train"]:  # reads q, k, v, dO, dhT (and h0), writes dq, dk, dv, dh0
            b += n * (4 * Hk + 3 * Hv) * rows + state * (3 if case["h0"] else 2)
            f += 10 * D * D * n * Hv
        return {"bytes": b, "flops": f}
    if op in ("decay_step", "delta_step"):
        R, Hk, Hv = case["rows"], case["Hk"], case["Hv"]
        return {"bytes": 2 * R * Hv * D * D * 4 + R * (2 * Hk + 2 * Hv) * 2 * D,
                "flops": R * Hv * D * D * (5 if op == "decay_step" else 9)}
    ql, kl, Hq, Hk = _ints(case["q"]), _key_lens(case), case["Hq"], case["Hk"]
    nq, nk = sum(ql), sum(kl)
    pairs = sum(_pairs(a, b) for a, b in zip(ql, kl))
    b = nq * Hq * (4 * D + 4) + nk * Hk * 4 * D
    f = 4 * D * pairs * Hq
    if case["train"]:  # reads q, k, v, o, lse, dO, writes dq, dk, dv
        b += nq * Hq * (8 * D + 4) + nk * Hk * 8 * D
        f += 10 * D * pairs * Hq
    return {"bytes": b, "flops": f}


def _pairs(q, k):
    """(query, key) pairs that the causal mask leaves: query i sees keys j <= i + k - q."""
    first = max(0, q - k)          # rows before this one see nothing
    n = q - first
    return n * (k - q + first + 1) + n * (n - 1) // 2 if n > 0 else 0


# ---- inputs ---------------------------------------------------------------------------------------------

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    bf = torch.bfloat16

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def unit(*shape):
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-20)).to(bf)

    def starts(lens):
        return torch.tensor([0] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)

    s = dict(case)
    op = case["op"]
    if op in ("decay", "decay_step"):
        # slow to fast heads: the slopes 2^(-8 (h + 1) / Hv), from 0.84 to 0.004 at 32 heads
        Hv = case["Hv"]
        s["decay"] = -torch.exp2(-8.0 * torch.arange(1, Hv + 1, device=dev, dtype=torch.float32) / Hv)
    if op == "decay":
        lens = _ints(case["lens"])
        n, Hk, Hv = sum(lens), case["Hk"], case["Hv"]
        s["cu"], s["max"] = starts(lens), max(lens)
        s["tq"], s["tk"], s["tv"] = unit(n, Hk, D), unit(n, Hk, D), normal(n, Hv, D).to(bf)
        s["th0"] = normal(len(lens), Hv, D, D) * 0.1 if case["h0"] else None
        if case["train"]:
            s["tdo"], s["tdhT"] = normal(n, Hv, D).to(bf), normal(len(lens), Hv, D, D) * 0.1
        return s
    if op in ("decay_step", "delta_step"):
        R, Hk, Hv = case["rows"], case["Hk"], case["Hv"]
        s["tq"], s["tk"], s["tv"] = unit(R, Hk, D), unit(R, Hk, D), normal(R, Hv, D).to(bf)
        s["state"] = normal(case["slots"], Hv, D, D) * 0.1
        s["at"] = torch.randperm(case["slots"], generator=gen, device=dev)[:R].to(torch.int32)
        if op == "delta_step":
            s["g"] = -torch.nn.functional.softplus(normal(R, Hv) + 1.0)
            s["beta"] = torch.sigmoid(normal(R, Hv))
        return s
    ql, kl, cap = _ints(case["q"]), _key_lens(case), case["cap"]
    Hq, Hk = case["Hq"], case["Hk"]
    nq, nk = sum(ql), (cap * len(kl) if cap else sum(kl))
    s["cu_q"], s["max_q"], s["max_k"] = starts(ql), max(ql), max(kl)
    # packed keys, or a cache of `cap` rows for each sequence, filled as far as k_len
    s["cu_k"] = starts([cap] * len(kl) if cap else kl)
    s["k_len"] = torch.tensor(kl, dtype=torch.int32).to(dev) if cap else None
    s["tq"], s["tk"], s["tv"] = normal(nq, Hq, D).to(bf), normal(nk, Hk, D).to(bf), normal(nk, Hk, D).to(bf)
    if case["train"]:
        s["tdo"] = normal(nq, Hq, D).to(bf)
    return s


# ---- one pass -------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"decay": _plain_decay, "decay_step": _plain_step, "delta_step": _plain_step, "attn": _plain_attn}[s["op"]](s)


def _run_own(s):
    import linear_attention_rnn_gb300 as gdn

    op = s["op"]
    if op == "decay":
        o, hT = gdn.decay_fwd(s["tq"], s["tk"], s["tv"], s["decay"], s["th0"], cu_seqlens=s["cu"], max_seqlen=s["max"])
        if not s["train"]:
            return {"o": o, "hT": hT}
        dq, dk, dv, dh0 = gdn.decay_bwd(s["tq"], s["tk"], s["tv"], s["decay"], s["th0"], s["tdo"], s["tdhT"],
                                        cu_seqlens=s["cu"], max_seqlen=s["max"])
        return {"o": o, "hT": hT, "dq": dq, "dk": dk, "dv": dv, "dh0": dh0}
    if op == "decay_step":
        return {"o": gdn.decay_step(s["tq"], s["tk"], s["tv"], s["decay"], s["state"], s["at"]), "state": s["state"]}
    if op == "delta_step":
        return {"o": gdn.delta_step(s["tq"], s["tk"], s["tv"], s["g"], s["beta"], s["state"], s["at"]), "state": s["state"]}
    o, lse = gdn.attn_fwd(s["tq"], s["tk"], s["tv"], cu_q=s["cu_q"], cu_k=s["cu_k"], k_len=s["k_len"], max_q=s["max_q"],
                          max_k=s["max_k"])
    if not s["train"]:
        return {"o": o, "lse": lse}
    dq, dk, dv = gdn.attn_bwd(s["tq"], s["tk"], s["tv"], o, lse, s["tdo"], cu_q=s["cu_q"], cu_k=s["cu_k"], max_q=s["max_q"],
                              max_k=s["max_k"])
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _padded(x, cu, lens, L):
    """Packed rows [N, H, D] as [n, H, L, D] in 32 bits, zero past each sequence's length."""
    t = torch.arange(L, device=x.device)
    inside = t[None, :] < lens[:, None]
    at = (cu[:-1, None].long() + t[None, :]).clamp_max(max(x.shape[0] - 1, 0))
    rows = torch.where(inside[:, :, None, None], x[at].float(), 0.0)
    return rows.permute(0, 2, 1, 3)


def _packed(y, cu, lens, total):
    """The first lens[b] rows of [n, H, L, D], one sequence behind another: [total, H, D]."""
    row = torch.arange(total, device=y.device)
    b = torch.searchsorted(cu[1:].long(), row, right=True)
    return y.permute(0, 2, 1, 3)[b, row - cu[b].long()]


def _flip(x, lens):
    """Each sequence's rows in reverse order: row t becomes row len - 1 - t."""
    t = torch.arange(x.shape[2], device=x.device)
    at = lens[:, None].long() - 1 - t[None, :]
    y = x.gather(2, at.clamp_min(0)[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3]))
    return torch.where((at >= 0)[:, None, :, None], y, 0.0)


def _linear(a, b, c, w, h0, lag):
    """o_t = sum over s <= t of e^(w (t - s)) (a_t . b_s) c_s, plus e^(w (t + lag)) h0^T a_t; [n, H, L, D] each."""
    n, H, L, _ = a.shape
    N = (L + CHUNK - 1) // CHUNK
    a_, b_, c_ = (torch.nn.functional.pad(x, (0, 0, 0, N * CHUNK - L)).reshape(n, H, N, CHUNK, D) for x in (a, b, c))
    i = torch.arange(CHUNK, device=a.device, dtype=torch.float32)
    gap = i[:, None] - i[None, :]
    mask = torch.where(gap >= 0, torch.exp(w[:, None, None] * gap.clamp_min(0)), 0.0)              # [H, C, C]
    o = ((a_ @ b_.transpose(-1, -2)) * mask[:, None]) @ c_
    u = (b_ * torch.exp(w[:, None] * (CHUNK - 1 - i))[:, None, :, None]).transpose(-1, -2) @ c_    # [n, H, N, D, D]
    m = torch.arange(N, device=a.device, dtype=torch.float32)
    hop = m[:, None] - 1 - m[None, :]
    carry = torch.where(hop >= 0, torch.exp(w[:, None, None] * CHUNK * hop.clamp_min(0)), 0.0)     # [H, N, N]
    enter = (carry @ u.reshape(n, H, N, D * D)).reshape(n, H, N, D, D)
    o = o + torch.exp(w[:, None] * (i + 1))[:, None, :, None] * (a_ @ enter)
    o = o.reshape(n, H, N * CHUNK, D)[:, :, :L]
    if h0 is not None:
        t = torch.arange(L, device=a.device, dtype=torch.float32)
        o = o + torch.exp(w[:, None] * (t + lag))[None, :, :, None] * (a @ h0)
    return o


def _plain_decay(s):
    q, k, v, w, h0, cu = s["tq"], s["tk"], s["tv"], s["decay"], s["th0"], s["cu"]
    total, L, G = q.shape[0], s["max"], s["Hv"] // s["Hk"]
    lens = cu[1:] - cu[:-1]
    Q, K = (_padded(x, cu, lens, L).repeat_interleave(G, 1) for x in (q, k))
    V = _padded(v, cu, lens, L)
    t = torch.arange(L, device=q.device, dtype=torch.float32)
    o = _linear(Q, K, V, w, h0, 1)
    left = (lens[:, None].float() - 1 - t).clamp_min(0)                       # steps from t to the last token
    hT = (K * torch.exp(w[None, :, None] * left[:, None, :])[..., None]).transpose(-1, -2) @ V
    all_of_it = torch.exp(w[None, :] * lens[:, None].float())[..., None, None]
    if h0 is not None:
        hT = hT + all_of_it * h0
    out = {"o": _packed(o, cu, lens, total).to(v.dtype), "hT": hT}
    if not s["train"]:
        return out
    dO, dhT = _padded(s["tdo"], cu, lens, L), s["tdhT"]
    n, Hk = lens.shape[0], s["Hk"]
    h0t = h0.transpose(-1, -2) if h0 is not None else None
    dq = _linear(dO, V, K, w, h0t, 1)
    Qr, Kr, Vr, dOr = (_flip(x, lens) for x in (Q, K, V, dO))
    dk = _flip(_linear(Vr, dOr, Qr, w, dhT.transpose(-1, -2), 0), lens)
    dv = _flip(_linear(Kr, Qr, dOr, w, dhT, 0), lens)
    dq, dk = (x.reshape(n, Hk, G, L, D).sum(2) for x in (dq, dk))
    dh0 = (Q * torch.exp(w[:, None] * (t + 1))[None, :, :, None]).transpose(-1, -2) @ dO + all_of_it * dhT
    out.update({"dq": _packed(dq, cu, lens, total).to(q.dtype), "dk": _packed(dk, cu, lens, total).to(k.dtype),
                "dv": _packed(dv, cu, lens, total).to(v.dtype), "dh0": dh0})
    return out


def _plain_step(s):
    G = s["Hv"] // s["Hk"]
    q, k = (s[x].float().repeat_interleave(G, 1) for x in ("tq", "tk"))       # [R, Hv, D]
    v, at = s["tv"].float(), s["at"].long()
    h = s["state"][at]
    if s["op"] == "decay_step":
        h = torch.exp(s["decay"])[None, :, None, None] * h + k[..., :, None] * v[..., None, :]
    else:
        h = torch.exp(s["g"])[..., None, None] * h
        new = s["beta"][..., None] * (v - (k[..., None, :] @ h)[..., 0, :])
        h = h + k[..., :, None] * new[..., None, :]
    s["state"][at] = h
    return {"o": (q[..., None, :] @ h)[..., 0, :].to(s["tv"].dtype), "state": s["state"]}


def _plain_attn(s):
    q, k, v, cu_q, cu_k = s["tq"], s["tk"], s["tv"], s["cu_q"], s["cu_k"]
    ql = cu_q[1:] - cu_q[:-1]
    kl = s["k_len"] if s["k_len"] is not None else cu_k[1:] - cu_k[:-1]
    Lq, Lk, G, n = s["max_q"], s["max_k"], s["Hq"] // s["Hk"], ql.shape[0]
    scale = 1.0 / math.sqrt(D)
    Q = _padded(q, cu_q, ql, Lq)                                              # [n, Hq, Lq, D]
    K, V = (_padded(x, cu_k, kl, Lk).repeat_interleave(G, 1) for x in (k, v))
    i, j = torch.arange(Lq, device=q.device), torch.arange(Lk, device=q.device)
    seen = (j[None, None, :] < kl[:, None, None]) & (j[None, None, :] <= i[None, :, None] + (kl - ql)[:, None, None])
    seen = seen[:, None]
    z = (Q @ K.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total == 0, 1.0, total))
    o = p @ V
    lse = (top + torch.log(total))
    out = {"o": _packed(o, cu_q, ql, q.shape[0]).to(q.dtype), "lse": _packed(lse, cu_q, ql, q.shape[0])[..., 0]}
    if not s["train"]:
        return out
    dO = _padded(s["tdo"], cu_q, ql, Lq)
    dv = p.transpose(-1, -2) @ dO
    ds = (dO @ V.transpose(-1, -2)).sub_((dO * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq, dk = ds @ K, ds.transpose(-1, -2) @ Q
    dk, dv = (x.reshape(n, s["Hk"], G, Lk, D).sum(2) for x in (dk, dv))
    out.update({"dq": _packed(dq, cu_q, ql, q.shape[0]).to(q.dtype), "dk": _packed(dk, cu_k, kl, k.shape[0]).to(k.dtype),
                "dv": _packed(dv, cu_k, kl, v.shape[0]).to(v.dtype)})
    return out


# ---- the definitions in 64 bits -------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attn":
        return _exact_attn(s, case)
    if op == "decay":
        return _exact_decay(s, case)
    f = lambda x: x.double()  # noqa: E731
    state = f(s["state"]).clone()
    o = torch.empty(s["tv"].shape, dtype=torch.float64, device="cuda")
    G = case["Hv"] // case["Hk"]
    for r, slot in enumerate(s["at"].tolist()):
        q, k, v, h = (f(x) for x in (s["tq"][r], s["tk"][r], s["tv"][r], state[slot]))
        q, k = (x.repeat_interleave(G, 0) for x in (q, k))
        if op == "decay_step":
            h = f(s["decay"]).exp()[:, None, None] * h + torch.einsum("hi,hj->hij", k, v)
        else:
            kh = torch.einsum("hi,hij->hj", k, h)
            a, b = f(s["g"][r]).exp()[:, None, None], f(s["beta"][r])[:, None, None]
            h = a * (h - b * torch.einsum("hi,hj->hij", k, kh)) + b * torch.einsum("hi,hj->hij", k, v)
        state[slot] = h
        o[r] = torch.einsum("hij,hi->hj", h, q)
    return {"o": o, "state": state}


def _exact_decay(s, case):
    """Token by token, all sequences side by side: the recurrence, and for the gradients its adjoint."""
    f = lambda x: None if x is None else x.double()  # noqa: E731
    lens, Hv, G = _ints(case["lens"]), case["Hv"], case["Hv"] // case["Hk"]
    q, k, v = f(s["tq"]).repeat_interleave(G, 1), f(s["tk"]).repeat_interleave(G, 1), f(s["tv"])
    keep = f(s["decay"]).exp()[None, :, None, None]
    start = s["cu"].tolist()
    hT = torch.zeros(len(lens), Hv, D, D, dtype=torch.float64, device="cuda")
    if s["th0"] is not None:
        hT = hT + f(s["th0"])
    o = torch.zeros_like(v)
    train = case["train"]
    dO = f(s["tdo"]) if train else None
    dq = torch.zeros_like(q) if train else None
    order = sorted(range(len(lens)), key=lambda b: -lens[b])   # the longest first: those alive at t are a prefix
    h = hT[order]
    base = [start[b] for b in order]
    for t in range(max(lens)):
        n = sum(x > t for x in lens)
        at = torch.tensor([base[b] + t for b in range(n)], device="cuda") if n > 1 else slice(base[0] + t, base[0] + t + 1)
        h[:n] = keep * h[:n] + k[at][..., :, None] * v[at][..., None, :]
        o[at] = (h[:n] * q[at][..., :, None]).sum(-2)
        if train:
            dq[at] = (h[:n] * dO[at][..., None, :]).sum(-1)
    hT[order] = h
    if not train:
        return {"o": o, "hT": hT}
    r = f(s["tdhT"])[order]
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for t in range(max(lens) - 1, -1, -1):
        n = sum(x > t for x in lens)
        at = torch.tensor([base[b] + t for b in range(n)], device="cuda") if n > 1 else slice(base[0] + t, base[0] + t + 1)
        r[:n] += q[at][..., :, None] * dO[at][..., None, :]
        dk[at] = (r[:n] * v[at][..., None, :]).sum(-1)
        dv[at] = (r[:n] * k[at][..., :, None]).sum(-2)
        r[:n] *= keep
    dh0 = torch.empty_like(r)
    dh0[order] = r
    fold = lambda x: x.reshape(x.shape[0], case["Hk"], G, D).sum(2)  # noqa: E731
    return {"o": o, "hT": hT, "dq": fold(dq), "dk": fold(dk), "dv": dv, "dh0": dh0}


def _exact_attn(s, case):
    """Sequence by sequence and head by head."""
    ql, kl, Hq, Hk, train = _ints(case["q"]), _key_lens(case), case["Hq"], case["Hk"], case["train"]
    if sum(a * b for a, b in zip(ql, kl)) * Hq > 5e9:   # (the widest products: some ten seconds)
        return None
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    d = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(sum(ql), Hq, D, **d), torch.full((sum(ql), Hq), -math.inf, **d)
    dq, dk, dv = torch.zeros(sum(ql), Hq, D, **d), torch.zeros(sum(kl), Hk, D, **d), torch.zeros(sum(kl), Hk, D, **d)
    for b, (n, m) in enumerate(zip(ql, kl)):
        if n == 0 or m == 0:
            continue
        hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1)
        for h in range(Hq):
            kh = h * Hk // Hq
            rows, keys = slice(cq[b], cq[b] + n), slice(ck[b], ck[b] + m)
            Q, K, V = s["tq"][rows, h].double(), s["tk"][keys, kh].double(), s["tv"][keys, kh].double()
            z = (Q @ K.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
            l = torch.logsumexp(z, 1)
            lse[rows, h] = l
            p = torch.exp(z - torch.where(l == -math.inf, 0.0, l)[:, None])
            out = p @ V
            o[rows, h] = out
            if train:
                dO = s["tdo"][rows, h].double()
                dv[keys, kh] += p.T @ dO
                ds = p * (dO @ V.T - (dO * out).sum(1, keepdim=True)) / math.sqrt(D)
                dq[rows, h] = ds @ K
                dk[keys, kh] += ds.T @ Q
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if train else {"o": o, "lse": lse}
