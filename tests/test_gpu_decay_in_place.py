"""Decayed linear attention that replaces its entering states: hT over h0, dh0 over dhT.

The same sums in the same order as with states of their own, so the results are equal bit for bit.
"""
import pytest
import torch

import test_gpu_decay as D

pytestmark = pytest.mark.gpu

# lengths, max_seqlen: the final states beside the walk in its launch, in one of their own (one
# segment, with and without enough CTAs to fill the GPU), behind segments, empty sequences, none but empty ones
CASES = [([300, 1, 65, 0], 300, 2), ([1500, 40, 0, 900], 1, 2), ([140] * 40 + [0], 140, 8), ([2600, 0, 130], 2600, 2),
         ([0, 700, 0], 1, 2), ([0, 0], 0, 2)]


def inputs(lens, Hv, seed):
    x = {k: t.cuda() for k, t in D.make(lens, 1, Hv, seed=seed).items()}
    return x, dict(cu_seqlens=D.cu(lens))


@pytest.mark.parametrize("lens,most,Hv", CASES)
def test_final_states_over_entering_ones(gdn_lib, lens, most, Hv):
    x, args = inputs(lens, Hv, 51)
    h = x["h0"].clone()
    ref = h.clone()
    for _ in range(3):  # a prompt read in parts goes on from its own states
        ro, ref = gdn_lib.decay_fwd(x["q"], x["k"], x["v"], x["decay"], ref, max_seqlen=most, **args)
        o, hT = gdn_lib.decay_fwd(x["q"], x["k"], x["v"], x["decay"], h, hT=h, max_seqlen=most, **args)
        assert hT is h
        assert torch.equal(o, ro) and torch.equal(h, ref)


@pytest.mark.parametrize("lens,most,Hv", CASES)
def test_gradients_over_the_cotangents_of_final_states(gdn_lib, lens, most, Hv):
    x, args = inputs(lens, Hv, 52)
    n, total, p = len(lens), sum(lens), lambda t: t.data_ptr()
    ref = gdn_lib.decay_bwd(x["q"], x["k"], x["v"], x["decay"], x["h0"], x["dO"], x["dhT"], max_seqlen=most, **args)
    need = gdn_lib.decay_workspace_bytes(1, n, total, most, 1, Hv)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    dq, dk, dv = (torch.empty_like(x[n_]) for n_ in ("q", "k", "v"))
    d = x["dhT"].clone()
    rc = gdn_lib.lib().gdn_decay_bwd(p(x["q"]), p(x["k"]), p(x["v"]), p(x["decay"]), p(x["h0"]), p(x["dO"]), p(d),
                                     p(args["cu_seqlens"]), p(dq), p(dk), p(dv), p(d), n, total, most, 1, Hv, 128, 128, 128,
                                     128, Hv * 128, p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    for a, b in zip((dq, dk, dv, d), ref):
        assert torch.equal(a, b)
    if total:
        assert gdn_lib.workspace_status(ws) == 0
