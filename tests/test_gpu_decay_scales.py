"""Decay passes of inputs far from one, for decays on both sides of where the masks' form changes.

The operation is linear in q, k, v and dO, so scaling them scales the results; nothing on the way may
leave fp32's range where the result does not.  Bounds: those of the decay tests, element by element.
"""
import pytest
import torch

import test_gpu_decay as D

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[300, 1, 65], [130]])
@pytest.mark.parametrize("scale", [1e-6, 1.0, 1e4])
@pytest.mark.parametrize("decays", [(-2.0, -2.4, -2.45, -2.49), (-2.51, -0.5, -1.2, -3.0)])
def test_scaled_inputs(gdn_lib, lens, scale, decays):
    x = D.make(lens, 2, 4, seed=41, h0=False)
    x["decay"] = torch.tensor(decays)
    for n in ("q", "k", "v", "dO"):
        x[n] = (x[n].float() * scale).bfloat16()
    x["dhT"] = x["dhT"] * scale ** 2  # (as a state is: a product of two)
    d = {k: None if t is None else t.cuda() for k, t in x.items()}
    args = dict(cu_seqlens=D.cu(lens), max_seqlen=max(lens))
    o, hT = gdn_lib.decay_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], **args)
    got = gdn_lib.decay_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["dO"], d["dhT"], **args)
    D.check_fwd(gdn_lib, x, lens, o, hT)
    D.check_bwd(gdn_lib, x, lens, got)


@pytest.mark.parametrize("decay", [-2.3, -2.49])
@pytest.mark.parametrize("size", [1e-12, 1e-11, 1e6, 1e10])
def test_diagonal_entries_of_any_size(gdn_lib, decay, size):
    """One pair of rows a token apart from the next: each output is its own token's product
    (a_t . b_t) c_t, but for what e^decay leaves of the token before.  Far from fp32's ends, so
    the bound is the decay tests' one, of each element."""
    T = 128
    gen = torch.Generator().manual_seed(42)
    row = torch.randn(T, 1, 128, generator=gen)
    unit = row / row.norm(dim=-1, keepdim=True)
    x = dict(q=unit.bfloat16(), k=(unit * size).bfloat16(), v=torch.randn(T, 1, 128, generator=gen).bfloat16(),
             decay=torch.tensor([decay]), h0=None, dO=torch.randn(T, 1, 128, generator=gen).bfloat16(),
             dhT=torch.zeros(1, 1, 128, 128))
    y = dict(x, q=(x["v"].float() * size).bfloat16(), v=x["q"], k=x["dO"], dO=x["k"])  # v . dO and k . q of that size
    for z in (x, y):
        d = {k: None if t is None else t.cuda() for k, t in z.items()}
        args = dict(cu_seqlens=D.cu([T]), max_seqlen=T)
        o, hT = gdn_lib.decay_fwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], **args)
        got = gdn_lib.decay_bwd(d["q"], d["k"], d["v"], d["decay"], d["h0"], d["dO"], d["dhT"], **args)
        D.check_fwd(gdn_lib, z, [T], o, hT)
        D.check_bwd(gdn_lib, z, [T], got)
