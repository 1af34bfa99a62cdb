"""Head counts for which a warp of rope_append holds keys beside values, or queries beside both:
against rope_fwd of the same rows, whose values the 64-bit definition bounds."""
import pytest
import torch

from oracle import ops
from test_gpu_rope import EPS, close, cuda, layout, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 1), (4, 1), (8, 1), (4, 2), (8, 2), (16, 2), (6, 3), (5, 5), (16, 4)])
@pytest.mark.parametrize("norms", ["both", "q", "k"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_keys_beside_values(gdn_lib, Hq, Hk, norms, interleaved):
    n, page = 301, 32
    x = make(n, Hq, Hk, 64, seed=Hq + Hk)
    if norms != "both":
        x["wk" if norms == "q" else "wq"] = None
    x["v"][::7] = float("nan")      # (values pass as they are, and touch no key)
    d = cuda(x)
    how = dict(q_weight=d["wq"], k_weight=d["wk"], eps=EPS, interleaved=interleaved)
    P = n // page + 3
    kp, vp = layout("rows", P, page, Hk)
    slots = torch.randperm(P * page, generator=torch.Generator().manual_seed(n))[:n].int()
    slots[5] = -1
    keep = slots >= 0
    to = slots[keep].long()
    wantk, wantv = kp.view(-1, Hk, 128).clone(), vp.view(-1, Hk, 128).clone()
    q0, k0 = gdn_lib.rope_fwd(d["q"], d["k"], d["pos"], d["freq"], **how)
    wantk[to.cuda()], wantv[to.cuda()] = k0[keep.cuda()], d["v"][keep.cuda()]
    q = gdn_lib.rope_append(d["q"], d["k"], d["v"], d["pos"], d["freq"], kp, vp, slots.cuda(), **how)
    angle = ops.angles(x["pos"], x["freq"])
    close(q, *ops.rope(x["q"], x["wq"], angle, interleaved, EPS), "q")
    bits = lambda t: t.flatten().view(torch.int16)
    assert torch.equal(bits(q), bits(q0))
    assert torch.equal(bits(kp), bits(wantk)) and torch.equal(bits(vp), bits(wantv))
