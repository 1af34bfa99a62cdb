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


# ---- heads' norms and rotation ------------------------------------------------------------
def _pairs(P, interleaved):
    first = torch.arange(P) * (2 if interleaved else 1)
    return first, first + (1 if interleaved else P)


def _turn(x, angle, interleaved):
    """x [n, H, d] with pair j of token t turned by angle[t, j]; and, of each value, the sizes that it is formed of."""
    i, j = _pairs(angle.shape[1], interleaved)
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    y, size = x.clone(), x.abs()
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    size[..., i] = size[..., j] = x[..., i].abs() + x[..., j].abs()
    return y, size


def angles(positions, freq, axis=None):
    """[n, P] from positions [n] or [axes, n], frequencies [P] and the axis of each pair."""
    pos = _d(positions).reshape(-1, positions.shape[-1])
    axis = torch.tensor(axis if axis is not None else [0] * freq.numel(), dtype=torch.long)
    return pos[axis].T * _d(freq)


def rope(x, w, angle, interleaved, eps):
    """(y, bound of its error): heads normed with weight w (None: not) and turned, in an evaluation
    in 32 bits that rounds the result once to bf16."""
    x, w = _d(x), _d(w)
    n = x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w
    y, size = _turn(n, angle, interleaved)
    # 32-bit roundings: 16 of 2^-24 for the norm (a sum of 128 squares in chains of 19, its root, two
    # products), 5e-7 for the angle, its cosine and sine, 3 for the turn
    return y, 2.0 ** -8 * y.abs() + 2e-6 * size


def rope_bwd(x, w, angle, interleaved, eps, dy):
    """(dx, its bound, dw, its bound)"""
    x, w, dy = _d(x), _d(w), _d(dy)
    dn, size = _turn(dy, -angle, interleaved)
    if w is None:
        return dn, 2.0 ** -8 * dn.abs() + 2e-6 * size, None, None
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    u, g = x * r, dn * w
    dx = r * (g - u * (g * u).mean(-1, keepdim=True))
    part = r * (size * w.abs() + u.abs() * (size * w.abs() * u.abs()).mean(-1, keepdim=True))
    rows = x.shape[0] * x.shape[1]
    # the sum over rows: chains of at most rows / 32 additions and 16 across threads
    dw_tol = (3e-6 + (16 + rows / 32) * 2.0 ** -24) * (size * u.abs()).sum((0, 1))
    return dx, 2.0 ** -8 * dx.abs() + 5e-6 * part, (dn * u).sum((0, 1)), dw_tol


# ---- keys in pages ------------------------------------------------------------------------
def rows_of(table, m, page, n_pages):
    """Flat rows (page * page_size + row) of a sequence's first m keys; -1 on absent pages."""
    rows = []
    for j in range(m):
        e = int(table[j // page])
        rows.append(e * page + j % page if 0 <= e < n_pages else -1)
    return rows


def _present(table, m, page, n_pages):
    rows = torch.tensor(rows_of(table, m, page, n_pages), dtype=torch.long)
    return torch.arange(m)[rows >= 0], rows[rows >= 0]


def attn_paged(q, k_pages, v_pages, table, ql, kl, scale, eps=0.0):
    """A dict of o and lse with their bounds (as attn), keys by page table [n][pages]."""
    q, kp, vp = _d(q), _d(k_pages), _d(v_pages)
    P, page, Hk, d = kp.shape
    G, u = q.shape[1] // Hk, 2.0 ** -8
    r = {"o": torch.zeros_like(q), "o_tol": torch.zeros_like(q),
         "lse": torch.full(q.shape[:2], -math.inf, dtype=torch.float64),
         "lse_tol": torch.zeros(q.shape[:2], dtype=torch.float64)}
    q0 = _starts(ql)
    for s, (n, m) in enumerate(zip(ql, kl)):
        at, flat = _present(table[s], m, page, P)
        if n == 0 or at.numel() == 0:
            continue
        hidden = at[None, :] > torch.arange(n)[:, None] + m - n
        rows = slice(q0[s], q0[s] + n)
        for h in range(q.shape[1]):
            K, V = kp.reshape(-1, Hk, d)[flat, h // G], vp.reshape(-1, Hk, d)[flat, h // G]
            z = (scale * (q[rows, h] @ K.T)).masked_fill(hidden, -math.inf)
            lse = torch.logsumexp(z, 1)
            p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[:, None])
            o, A = p @ V, p @ V.abs()
            r["o"][rows, h], r["o_tol"][rows, h] = o, u * o.abs() + (u + 2 * eps) * A
            r["lse"][rows, h], r["lse_tol"][rows, h] = lse, eps + (m + 256) * 2.0 ** -23
    return r


def attn_paged_weights(q, k_pages, lse, table, ql, kl, weights, scale, eps=0.0):
    """(weights, bound of their error): what each key receives added to its place."""
    q, kp, lse, w = _d(q), _d(k_pages), _d(lse), _d(weights).clone()
    P, page, Hk, d = kp.shape
    G = q.shape[1] // Hk
    tol = torch.zeros_like(w)
    q0 = _starts(ql)
    for s, (n, m) in enumerate(zip(ql, kl)):
        at, flat = _present(table[s], m, page, P)
        if n == 0 or at.numel() == 0:
            continue
        hidden = at[None, :] > torch.arange(n)[:, None] + m - n
        for h in range(q.shape[1]):
            rows, kh = slice(q0[s], q0[s] + n), h // G
            l = lse[rows, h, None]
            z = scale * (q[rows, h] @ kp.reshape(-1, Hk, d)[flat, kh].T)
            p = torch.where(hidden | (l == -math.inf), 0.0, torch.exp(z - l))
            # of each term: the score, the exponent's two roundings, ex2; and chains of at most 64 + n G / 128
            # additions (a query tile's terms in four, 32 each, or 16; then tile by tile, joins)
            off = p * (eps + (z.abs() + torch.where(l.isinf(), 0.0, l.abs())) * 2.0 ** -22 + 2.0 ** -21
                       + (64 + n * G / 128) * 2.0 ** -24)
            for x, y in ((w, p), (tol, off)):
                x.view(P, Hk, page).index_put_((flat // page, torch.full_like(flat, kh), flat % page), y.sum(0),
                                               accumulate=True)
    return w, tol + 2.0 ** -22 * w.abs()


def cache_evict(k_pages, v_pages, weights, table, kl, budget, recent, to):
    """(k_pages, v_pages, weights, new lengths), the first three in their own types: by sorting."""
    kp, vp, w = (x.detach().cpu() for x in (k_pages, v_pages, weights))
    P, page, Hk, _ = kp.shape
    nk, nv, nw, new = kp.clone(), vp.clone(), w.clone(), []
    for s, m in enumerate(kl):
        rows, target = rows_of(table[s], m, page, P), rows_of(to[s], min(m, len(to[s]) * page), page, P)
        old = m - min(recent, budget, m)
        last = [j for j in range(old, m) if rows[j] >= 0]
        some = [j for j in range(old) if rows[j] >= 0]
        take = min(len(some), budget - len(last))
        new.append(take + len(last))
        for h in range(Hk):
            weight = {j: float(w[rows[j] // page, h, rows[j] % page]) for j in some}
            key = lambda j: -math.inf if math.isnan(weight[j]) else weight[j]
            # (NaN below minus infinity)
            order = sorted(some, key=lambda j: (math.isnan(weight[j]), -key(j), j))
            for i, j in enumerate(sorted(order[:take]) + last):
                if target[i] < 0:
                    continue
                a, b = divmod(rows[j], page), divmod(target[i], page)
                nk[b[0], b[1], h], nv[b[0], b[1], h] = kp[a[0], a[1], h], vp[a[0], a[1], h]
                nw[b[0], h, b[1]] = w[a[0], h, a[1]]
    return nk, nv, nw, new
