"""Workspaces at any multiple of 16 bytes give what aligned ones give, bit by bit."""
import pytest
import torch

import paged

pytestmark = pytest.mark.gpu


def place(nbytes, shift):
    """`nbytes` that begin `shift` bytes behind a multiple of 512, between guards."""
    whole = torch.full((nbytes + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    at = -whole.data_ptr() % 512 + shift
    ws = whole[at:at + nbytes]
    assert ws.data_ptr() % 512 == shift
    return whole, ws, at


def untouched(whole, ws, at):
    return bool((whole[:at] == 0xA5).all()) and bool((whole[at + ws.numel():] == 0xA5).all())


@pytest.mark.parametrize("shift", [0, 16, 48, 128 + 16])
@pytest.mark.parametrize("ql,kl,Hq,Hk", [
    ([1, 2, 1], [2999, 1500, 17], 4, 2),       # one query tile, items that are cut
    ([3], [20000], 6, 2),
    ([300, 5], [1300, 2000], 4, 2),            # several query tiles
])
def test_attention_and_weights(gdn_lib, ql, kl, Hq, Hk, shift):
    x = paged.cuda(paged.cache(ql, kl, Hq, Hk, 16, seed=sum(kl)))
    at = dict(cu_q=x["cu"], max_q=max(ql), max_k=max(kl))
    args = (x["q"], x["kp"], x["vp"], x["table"], x["k_len"])
    o, lse = gdn_lib.attn_paged(*args, **at)
    nbytes = gdn_lib.attn_paged_workspace_bytes(len(ql), sum(ql), x["table"].shape[1] * 16, max(ql), max(kl), Hq, Hk)
    assert nbytes > 256 * 1024                 # (parts are written)
    whole, ws, begin = place(nbytes, shift)
    o2, lse2 = gdn_lib.attn_paged(*args, workspace=ws, **at)
    assert gdn_lib.workspace_status(ws) == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and untouched(whole, ws, begin)
    w = gdn_lib.attn_paged_weights(x["q"], x["kp"], lse, x["table"], x["k_len"], x["weights"].clone(), **at)
    whole, ws, begin = place(256, shift)
    w2 = gdn_lib.attn_paged_weights(x["q"], x["kp"], lse, x["table"], x["k_len"], x["weights"].clone(), workspace=ws, **at)
    assert gdn_lib.workspace_status(ws) == 0 and torch.equal(w, w2) and untouched(whole, ws, begin)


@pytest.mark.parametrize("shift", [16, 48])
def test_eviction_and_rotation(gdn_lib, shift):
    x = paged.cuda(paged.cache([1, 1], [700, 90], 2, 2, 16, seed=3, nan=False))
    runs = []
    for given in (False, True):
        c = [x[n].clone() for n in ("kp", "vp", "weights")]
        whole, ws, begin = place(gdn_lib.cache_evict_workspace_bytes(2, x["table"].shape[1] * 16, 300, 2), shift)
        n = gdn_lib.cache_evict(*c, x["table"], x["k_len"], 300, recent=7, workspace=ws if given else None)
        assert untouched(whole, ws, begin)
        runs.append([*c, n])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    q, k, dq, dk = r(999, 4, 128), r(999, 2, 128), r(999, 4, 128), r(999, 2, 128)
    w = torch.ones(128, device="cuda")
    pos, freq = torch.arange(999, dtype=torch.int32, device="cuda"), torch.rand(64, generator=gen, device="cuda")
    whole, ws, begin = place(gdn_lib.rope_workspace_bytes(999, 4, 2), shift)
    runs = [gdn_lib.rope_bwd(q, k, pos, freq, dq, dk, q_weight=w, k_weight=w, workspace=t) for t in (None, ws)]
    assert all(torch.equal(a, b) for a, b in zip(*runs)) and untouched(whole, ws, begin)
