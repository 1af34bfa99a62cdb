"""The operators on a stream of their own, and as a captured graph replayed on new inputs.

A graph holds the same launches, so its results equal the plain calls' bit for bit.
"""
import pytest
import torch

import test_gpu_attn as A
import test_gpu_decay as D
import test_gpu_step as S

pytestmark = pytest.mark.gpu


def token(gdn, x):
    """One decoding step of each mixer: state or cache in, output out."""
    state1, state2 = x["state"].clone(), x["state"].clone()
    o1 = gdn.delta_step(x["q"], x["k"], x["v"], x["g"], x["beta"], state1, x["slots"])
    o2 = gdn.decay_step(x["q"], x["k"], x["v"], x["decay"], state2, x["slots"])
    o3, lse = gdn.attn_fwd(x["aq"], x["ak"], x["av"], cu_q=x["cu_q"], cu_k=x["cu_k"], k_len=x["k_len"], max_k=4000)
    return o1, o2, o3, lse, state1, state2


def train(gdn, x):
    """A training pass of the two mixers with a backward."""
    s = x["seq"]
    o, hT = gdn.decay_fwd(s["q"], s["k"], s["v"], s["decay"], s["h0"], cu_seqlens=x["cu"], max_seqlen=1900)
    d = gdn.decay_bwd(s["q"], s["k"], s["v"], s["decay"], s["h0"], s["dO"], s["dhT"], cu_seqlens=x["cu"], max_seqlen=1900)
    t = x["att"]
    ao, lse = gdn.attn_fwd(t["q"], t["k"], t["v"], cu_q=x["cu"], cu_k=x["cu"], max_k=1900)
    ad = gdn.attn_bwd(t["q"], t["k"], t["v"], ao, lse, t["dO"], cu_q=x["cu"], cu_k=x["cu"])
    return (o, hT, *d, ao, lse, *ad)


def inputs(seed):
    x = {k: t.cuda() for k, t in S._rows(5, 2, 4, 8, seed=seed).items()}
    a = A.make([1] * 3, [4000] * 3, 4, 2, seed=seed)
    x.update(aq=a["q"].cuda(), ak=a["k"].cuda(), av=a["v"].cuda(), cu_q=A.cu([1] * 3), cu_k=A.cu([4000] * 3),
             k_len=torch.tensor([4000, 0, 77 + seed], dtype=torch.int32).cuda())
    lens = [1900, 0, 333]
    x["cu"] = D.cu(lens)
    x["seq"] = {k: t.cuda() for k, t in D.make(lens, 1, 2, seed=seed).items()}
    x["att"] = {k: t.cuda() for k, t in A.make(lens, lens, 4, 2, seed=seed).items()}
    return x


def tensors(x):
    for t in x.values():
        if isinstance(t, dict):
            yield from t.values()
        else:
            yield t


@pytest.mark.parametrize("f", [token, train])
def test_side_stream(gdn_lib, f):
    x = inputs(1)
    plain = f(gdn_lib, x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = f(gdn_lib, x)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, plain))


@pytest.mark.parametrize("f", [token, train])
def test_captured_graph(gdn_lib, f):
    x = inputs(2)
    f(gdn_lib, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = f(gdn_lib, x)
    for seed in (3, 4):
        y = inputs(seed)
        for a, b in zip(tensors(x), tensors(y)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        plain = f(gdn_lib, y)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, plain))
