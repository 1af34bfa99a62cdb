"""64-bit restatements of the operators around the chunked rule, from their definitions.

Every function works on torch tensors of any floating type (widened exactly),
sequence by sequence and, for the recurrences, token by token.
"""
from __future__ import annotations

import math

import torch


def _d(x):
    return None if x is None else x.detach().cpu().double()


def delta_step(q, k, v, g, beta, state, slots):
    """(o, state): one token per row of the gated delta rule (rows with a slot
    below 0 have no state and give zero)."""
    q, k, v, g, beta, state = map(_d, (q, k, v, g, beta, state))
    state = state.clone()
    G = v.shape[1] // k.shape[1]
    o = torch.zeros_like(v)
    for r, s in enumerate(slots):
        if s < 0:
            continue
        for j in range(v.shape[1]):
            kk, qq, h = k[r, j // G], q[r, j // G], state[s, j]
            h = math.exp(g[r, j]) * (h - beta[r, j] * torch.outer(kk, kk @ h)) + beta[r, j] * torch.outer(kk, v[r, j])
            state[s, j] = h
            o[r, j] = qq @ h
    return o, state


def decay_step(q, k, v, decay, state, slots):
    q, k, v, decay, state = map(_d, (q, k, v, decay, state))
    state = state.clone()
    G = v.shape[1] // k.shape[1]
    o = torch.zeros_like(v)
    for r, s in enumerate(slots):
        if s < 0:
            continue
        for j in range(v.shape[1]):
            state[s, j] = math.exp(decay[j]) * state[s, j] + torch.outer(k[r, j // G], v[r, j])
            o[r, j] = q[r, j // G] @ state[s, j]
    return o, state


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def decay_fwd(q, k, v, decay, h0, lens):
    """(o, hT) of packed rows [total, H, D]: S_t = e^w S_{t-1} + k_t v_t^T, o_t = S_t^T q_t."""
    q, k, v, decay, h0 = map(_d, (q, k, v, decay, h0))
    Hv, G = v.shape[1], v.shape[1] // k.shape[1]
    q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    keep = torch.exp(decay)[:, None, None]
    o = torch.zeros_like(v)
    hT = torch.zeros(len(lens), Hv, k.shape[2], v.shape[2], dtype=torch.float64)
    at = _starts(lens)
    for s in range(len(lens)):
        h = h0[s].clone() if h0 is not None else hT[s]
        for t in range(at[s], at[s + 1]):
            h = keep * h + k[t][:, :, None] * v[t][:, None, :]
            o[t] = (q[t][:, None, :] @ h)[:, 0]
        hT[s] = h
    return o, hT


def decay_bwd(q, k, v, decay, h0, dO, dhT, lens):
    """(dq, dk, dv, dh0): the recurrence's adjoint, token by token."""
    q, k, v, decay, h0, dO, dhT = map(_d, (q, k, v, decay, h0, dO, dhT))
    Hk, Hv = k.shape[1], v.shape[1]
    G = Hv // Hk
    q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    keep = torch.exp(decay)[:, None, None]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dh0 = torch.zeros(len(lens), Hv, k.shape[2], v.shape[2], dtype=torch.float64)
    at = _starts(lens)
    for s in range(len(lens)):
        h = h0[s].clone() if h0 is not None else torch.zeros_like(dh0[s])
        for t in range(at[s], at[s + 1]):
            h = keep * h + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = (h @ dO[t][:, :, None])[:, :, 0]
        r = dhT[s].clone() if dhT is not None else torch.zeros_like(dh0[s])
        for t in range(at[s + 1] - 1, at[s] - 1, -1):
            r = r + q[t][:, :, None] * dO[t][:, None, :]
            dk[t] = (r @ v[t][:, :, None])[:, :, 0]
            dv[t] = (k[t][:, None, :] @ r)[:, 0]
            r = keep * r
        dh0[s] = r
    fold = lambda x: x.reshape(x.shape[0], Hk, G, x.shape[2]).sum(2)
    return fold(dq), fold(dk), dv, dh0


def attn(q, k, v, ql, k0, kl, scale, dO=None, eps=0.0):
    """Causal attention of packed sequences: ql queries each, keys k0[s] .. k0[s] + kl[s] - 1.
    Returns a dict of o, lse (and dq, dk, dv), each with the bound of its error, "<name>_tol",
    in an evaluation that keeps sums in 32 bits and rounds p, ds and every result once to bf16
    (unit roundoff 2^-8), with scores off by at most eps."""
    q, k, v, dO = map(_d, (q, k, v, dO))
    G = q.shape[1] // k.shape[1]
    u = 2.0 ** -8
    zero = lambda x: torch.zeros_like(x)
    r = {"o": zero(q), "o_tol": zero(q), "lse": torch.full(q.shape[:2], -math.inf, dtype=torch.float64),
         "lse_tol": torch.zeros(q.shape[:2], dtype=torch.float64)}
    if dO is not None:
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            r[n], r[n + "_tol"] = zero(x), zero(x)
    q0 = _starts(ql)
    for s, (n, m) in enumerate(zip(ql, kl)):
        if n == 0 or m == 0:
            continue
        rows, keys = slice(q0[s], q0[s] + n), slice(k0[s], k0[s] + m)
        hidden = torch.arange(m)[None, :] > torch.arange(n)[:, None] + m - n
        for h in range(q.shape[1]):
            Q, K, V = q[rows, h], k[keys, h // G], v[keys, h // G]
            z = (scale * (Q @ K.T)).masked_fill(hidden, -math.inf)
            lse = torch.logsumexp(z, 1)
            p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[:, None])
            o, A = p @ V, p @ V.abs()
            r["o"][rows, h], r["o_tol"][rows, h] = o, u * o.abs() + (u + 2 * eps) * A
            r["lse"][rows, h], r["lse_tol"][rows, h] = lse, eps + (m + 256) * 2.0 ** -23
            if dO is None:
                continue
            d = dO[rows, h]
            dp, delta = d @ V.T, (d * o).sum(1, keepdim=True)
            ds = scale * p * (dp - delta)
            off = (d.abs() * r["o_tol"][rows, h]).sum(1, keepdim=True)  # of delta, from the rounded o
            size = (u + 3 * eps) * ds.abs() + scale * p * (off + 256 * 2.0 ** -23 * (d.abs() @ V.abs().T))
            r["dq"][rows, h], r["dq_tol"][rows, h] = ds @ K, size @ K.abs()
            r["dk"][keys, h // G] += ds.T @ Q
            r["dk_tol"][keys, h // G] += size.T @ Q.abs()
            r["dv"][keys, h // G] += p.T @ d
            r["dv_tol"][keys, h // G] += (u + 3 * eps) * (p.T @ d.abs())
    if dO is not None:
        for n in ("dq", "dk", "dv"):
            r[n + "_tol"] += u * r[n].abs()
    return r
