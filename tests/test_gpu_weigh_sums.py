"""Long sums of key weights keep the bound that their roundings give.

All queries are equal, so that a key's weight is the count of its terms times one of them, and each addition of
a chain rounds the same way for whole binades of the sum: a chain of N equal terms is off by up to N 2^-25 of
its value.  The bound (as in oracle.ops.attn_paged_weights, of each term): the score's roundings eps, (|z| + |lse|)
2^-22 for the exponent's, 2^-21 for ex2, and chains of at most 64 + n G / 128 additions."""
import pytest
import torch

import paged
from test_gpu_attn import close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,more,Hq,Hk,most_q,seed", [
    (16384, 512, 16, 4, "exact", 1),     # a CTA to a key tile
    (16384, 512, 16, 4, "exact", 2),
    (16384, 512, 8, 1, "exact", 3),      # a pair of CTAs
    (5000, 640, 8, 1, "exact", 4),
    (4096, 512, 4, 1, 1, 5),             # a bound that is too small: the kernel for few rows
    (64, 4000, 16, 4, "exact", 6),       # what that kernel is for
])
def test_equal_terms(gdn_lib, n, more, Hq, Hk, most_q, seed):
    m, page, G = n + more, 64, Hq // Hk
    gen = torch.Generator().manual_seed(seed)
    scale = 128 ** -0.5
    pages = -(-m // page)
    # scores z = scale a b of one product each: a a power of two, b in bf16
    a, lse = 0.125, 0.4
    b = (torch.rand(pages * page, Hk, generator=gen) * 8).bfloat16()
    kp = torch.zeros(pages, page, Hk, 128, dtype=torch.bfloat16)
    kp[..., 0] = b.view(pages, page, Hk)
    q = torch.zeros(n, Hq, 128, dtype=torch.bfloat16)
    q[..., 0] = a
    w = gdn_lib.attn_paged_weights(q.cuda(), kp.cuda(), torch.full((n, Hq), lse).cuda(),
                                   torch.arange(pages, dtype=torch.int32).view(1, -1).cuda(), paged.ints([m]).cuda(),
                                   torch.zeros(pages, Hk, page).cuda(), cu_q=paged.cu([n]).cuda(),
                                   max_q=n if most_q == "exact" else most_q, max_k=m)
    got = w.cpu().transpose(1, 2).reshape(pages * page, Hk)[:more]        # (all queries see the first ones)
    z = scale * a * b[:more].double()
    lse = float(torch.tensor(lse))
    want = n * G * torch.exp(z - lse)
    eps = float(z.abs().max()) * 136 * 2.0 ** -23
    tol = want * (eps + (z.abs() + abs(lse)) * 2.0 ** -22 + 2.0 ** -21 + (64 + n * G / 128) * 2.0 ** -24 + 2.0 ** -22)
    worst = float(((got.double() - want).abs() / tol).max())
    print(f"n {n} heads {Hq}/{Hk}: {worst:.2f} of the bound, {float(((got.double() - want).abs() / want).max()):.1e} of the value")
    close(got, want, tol, "weights")
