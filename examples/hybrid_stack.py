"""A stack that alternates the three token mixers: the gated delta rule, linear attention
with a decay for each head, and causal softmax attention with grouped heads.

    python examples/hybrid_stack.py

Packed prompts of different lengths are read in one pass, tokens are then decoded
one by one for all sequences together (states updated in place, keys and values
appended to caches of fixed capacity), and the decoded outputs are compared with
those of one pass over the longer prompts.  A training pass returns the
gradients of every mixer's inputs.  Weights are random; the projections around
the mixers are plain matrix products of one fused buffer, whose parts the mixers
read where they lie.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_rnn_gb300 as gdn  # noqa: E402

D = 128  # head size


def unit(x):
    return torch.nn.functional.normalize(x.float(), dim=-1).to(x.dtype)


class Mixer:
    """q, k, v (and for the delta rule gate logits) as one projection of the hidden rows."""

    def __init__(self, kind, width, Hq, Hk, gen):
        self.kind, self.Hq, self.Hk = kind, Hq, Hk
        # the linear mixers share q and k among value heads, softmax attention k and v among query heads
        self.parts = [Hq * D, Hk * D, Hk * D] if kind == "attn" else [Hk * D, Hk * D, Hq * D]
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        self.w = (r(width, sum(self.parts)) * width ** -0.5).bfloat16()
        self.out = (r(Hq * D, width) * (Hq * D) ** -0.5).bfloat16()
        self.gates = r(width, 2 * Hq) * width ** -0.5 if kind == "delta" else None
        self.decay = -torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq)

    def split(self, x):
        q, k, v = (x @ self.w).split(self.parts, -1)
        q, k, v = (t.unflatten(-1, (-1, D)) for t in (q, k, v))
        if self.kind == "delta":  # the rule takes unit rows, contiguous
            return unit(q), unit(k), v.contiguous()
        return (q, k, v) if self.kind == "attn" else (unit(q), unit(k), v)

    def delta_gates(self, x):
        g, beta = (x.float() @ self.gates).chunk(2, -1)
        return -torch.nn.functional.softplus(g + 1.0).contiguous(), torch.sigmoid(beta).contiguous()

    def prompt(self, x, lens, cu, capacity):
        """(mixed rows, what the next tokens need): packed rows x of sequences of `lens` tokens."""
        q, k, v = self.split(x)
        if self.kind == "decay":
            o, state = gdn.decay_fwd(q, k, v, self.decay, cu_seqlens=cu, max_seqlen=max(lens))
            return o, state
        if self.kind == "attn":
            o, _ = gdn.attn_fwd(q, k, v, cu_q=cu, cu_k=cu, max_q=max(lens), max_k=max(lens))
            cache = [torch.zeros(len(lens), capacity, self.Hk, D, dtype=x.dtype, device=x.device) for _ in "kv"]
            for b, (ks, vs) in enumerate(zip(k.split(lens), v.split(lens))):
                cache[0][b, :lens[b]], cache[1][b, :lens[b]] = ks, vs
            return o, cache
        g, beta = self.delta_gates(x)
        o, state, at = torch.empty_like(v), [], 0
        for n in lens:  # (the delta rule's prompt pass takes sequences of one length)
            rows = [t[None, at:at + n] for t in (q, k, v, g, beta)]
            o[at:at + n], h = gdn.chunk_fwd(*rows)
            state.append(h)
            at += n
        return o, torch.cat(state)

    def token(self, x, state, used):
        """The next token of every sequence; `used`: int32 lengths including it."""
        q, k, v = self.split(x)
        if self.kind == "delta":
            return gdn.delta_step(q, k, v, *self.delta_gates(x), state)
        if self.kind == "decay":
            return gdn.decay_step(q, k, v, self.decay, state)
        rows = torch.arange(x.shape[0], device=x.device)
        state[0][rows, used.long() - 1], state[1][rows, used.long() - 1] = k, v
        return gdn.attn_fwd(q[:, None], *state, k_len=used, want_lse=False)[0][:, 0]


class Stack:
    def __init__(self, kinds=("delta", "decay", "attn"), width=512, Hq=8, Hk=4, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.width = width
        self.mixers = [Mixer(kind, width, Hq, Hk, gen) for kind in kinds]

    def prompt(self, x, lens, capacity):
        cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()
        states = []
        for m in self.mixers:
            o, s = m.prompt(x, lens, cu, capacity)
            states.append(s)
            x = x + o.flatten(-2) @ m.out
        return x, states

    def token(self, x, states, used):
        for m, s in zip(self.mixers, states):
            x = x + m.token(x, s, used).flatten(-2) @ m.out
        return x


def decode(lens, steps, seed=1, **kw):
    """Largest difference, over the largest output, of decoded tokens from one pass over all of them."""
    stack = Stack(**kw)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    whole = [torch.randn(n + steps, stack.width, generator=gen, device="cuda").bfloat16() for n in lens]
    ref, _ = stack.prompt(torch.cat(whole), [n + steps for n in lens], max(lens) + steps)
    ref = torch.stack([r[n:] for r, n in zip(ref.split([n + steps for n in lens]), lens)])
    _, states = stack.prompt(torch.cat([w[:n] for w, n in zip(whole, lens)]), list(lens), max(lens) + steps)
    used = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = []
    for t in range(steps):
        used += 1
        out.append(stack.token(torch.stack([w[n + t] for w, n in zip(whole, lens)]), states, used))
    out = torch.stack(out, 1)
    return float((out.float() - ref.float()).abs().max() / ref.float().abs().max())


def gradients(lens, seed=2, Hq=8, Hk=4):
    """One training pass of the decay and the softmax mixer over packed rows: outputs and the
    gradients of their inputs for random output cotangents."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda H: torch.randn(sum(lens), H, D, generator=gen, device="cuda").bfloat16()
    cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()
    w = -torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq)
    q, k, v, dO = unit(r(Hk)), unit(r(Hk)), r(Hq), r(Hq)
    o, hT = gdn.decay_fwd(q, k, v, w, cu_seqlens=cu, max_seqlen=max(lens))
    linear = (o,) + gdn.decay_bwd(q, k, v, w, None, dO, cu_seqlens=cu, max_seqlen=max(lens))
    q, k, v = r(Hq), r(Hk), r(Hk)
    o, lse = gdn.attn_fwd(q, k, v, cu_q=cu, cu_k=cu)
    softmax = (o,) + gdn.attn_bwd(q, k, v, o, lse, dO, cu_q=cu, cu_k=cu)
    return linear, softmax


def main():
    gdn.lib()
    lens, steps = (700, 1, 129, 384), 16
    print(f"decoded {steps} tokens behind prompts of {lens}: largest difference {decode(lens, steps):.1e} of the largest output")
    linear, softmax = gradients(lens)
    print("decay mixer: o", tuple(linear[0].shape), "dq", tuple(linear[1].shape), "dk", tuple(linear[2].shape),
          "dv", tuple(linear[3].shape))
    print("softmax mixer: o", tuple(softmax[0].shape), "dq", tuple(softmax[1].shape), "dk", tuple(softmax[2].shape),
          "dv", tuple(softmax[3].shape))


if __name__ == "__main__":
    main()
