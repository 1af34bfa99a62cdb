"""Pages whose heads are not the rows' size are refused: the library takes strides alone and moves 128
values of a head (CPU, operands on devices that are not there)."""
import types

import pytest
import torch

import linear_attention_rnn_gb300 as gdn
from test_paged_host import BF, CALLS, MODE, calls, operands  # noqa: F401  (calls: a fixture)


@pytest.mark.parametrize("call", ["rope_append", "attn_paged", "attn_paged_weights"])
@pytest.mark.parametrize("d", [64, 256])
def test_another_head_size(calls, call, d):  # noqa: F811
    x = operands(kp=(3, 16, 1, d, BF), vp=(3, 16, 1, d, BF))
    with MODE, pytest.raises(ValueError):
        CALLS[call][0](x)
    assert not calls


@pytest.mark.parametrize("call", ["rope_append", "attn_paged", "attn_paged_weights"])
def test_part_of_wider_heads(calls, call):  # noqa: F811
    """The first 64 values of heads of 128: their strides are those of whole ones."""
    x = operands()
    with MODE:
        x.kp, x.vp = x.kp[..., :64], x.vp[..., :64]
    with MODE, pytest.raises(ValueError):
        CALLS[call][0](x)
    assert not calls


def test_values_alone(calls):  # noqa: F811
    x = operands(vp=(3, 16, 1, 64, BF))
    with MODE, pytest.raises(ValueError):
        CALLS["rope_append"][0](x)
    assert not calls


def test_eviction_asks_the_library():
    """Its head size is the pages' own, which the library refuses where it is not 128."""
    seen = []
    lib = types.SimpleNamespace(gdn_cache_evict_workspace_bytes=lambda *a: 0,
                                gdn_cache_evict=lambda *a: seen.append(a[13]) or -2, gdn_strerror=lambda c: b"")
    x = operands(kp=(3, 16, 1, 64, BF), vp=(3, 16, 1, 64, BF))
    with pytest.MonkeyPatch.context() as m, MODE:
        m.setattr(gdn, "lib", lambda: lib)
        m.setattr(gdn, "_several_devices", False)
        m.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
        with pytest.raises(gdn.GDNError):
            gdn.cache_evict(x.kp, x.vp, x.weights, x.table, x.k_len, 9, new_len=x.new_len)
    assert seen == [64]
