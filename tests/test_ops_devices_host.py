"""Devices of the operators' operands, workspaces and cached sizes -- no GPU needed: the operands
are shapes on devices that are not there, the library is a stand-in."""
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import linear_attention_rnn_gb300 as gdn

MODE = FakeTensorMode(allow_non_fake_inputs=True)
BF, F, I = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture
def at(monkeypatch):
    """The current device, as a list of one index; a library whose answers depend on it and whose calls are counted."""
    at = [0]
    calls = []

    def stand_in(name):
        def f(*args):
            if name.endswith("workspace_bytes"):
                return 1000 * (at[0] + 1)
            calls.append(name)
            return 0
        f.__name__ = name
        return f
    L = types.SimpleNamespace(**{n: stand_in(n) for n in (
        "gdn_delta_step", "gdn_decay_step", "gdn_decay_fwd", "gdn_decay_bwd", "gdn_attn_fwd", "gdn_attn_bwd",
        "gdn_decay_workspace_bytes", "gdn_attn_workspace_bytes")})
    monkeypatch.setattr(gdn, "lib", lambda: L)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: at[0])
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(gdn, "_several_devices", True, raising=False)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)  # (shapes on devices make no context then)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    at.append(calls)
    return at


def operands(where, other, at):
    """Every operand of a call on device `where`, but `other` on device `at`."""
    shapes = dict(q=(4, 2, 128, BF), k=(4, 2, 128, BF), v=(4, 2, 128, BF), g=(4, 2, F), beta=(4, 2, F), w=(2, F),
                  state=(4, 2, 128, 128, F), slots=(4, I), o=(4, 2, 128, BF), dO=(4, 2, 128, BF), lse=(4, 2, F), cu=(2, I),
                  cu_k=(2, I), h0=(1, 2, 128, 128, F), hT=(1, 2, 128, 128, F), dhT=(1, 2, 128, 128, F), k_len=(1, I),
                  ws=(1 << 20, torch.uint8))
    with MODE:
        return types.SimpleNamespace(**{n: torch.empty(s[:-1], dtype=s[-1], device=f"cuda:{at if n == other else where}")
                                        for n, s in shapes.items()})


CALLS = {
    "delta_step": (lambda x: gdn.delta_step(x.q, x.k, x.v, x.g, x.beta, x.state, x.slots, o=x.o),
                   "q k v g beta state slots o"),
    "decay_step": (lambda x: gdn.decay_step(x.q, x.k, x.v, x.w, x.state, x.slots, o=x.o), "q k v w state slots o"),
    "decay_fwd": (lambda x: gdn.decay_fwd(x.q, x.k, x.v, x.w, x.h0, cu_seqlens=x.cu, o=x.o, hT=x.hT, workspace=x.ws),
                  "q k v w h0 cu o hT ws"),
    "decay_bwd": (lambda x: gdn.decay_bwd(x.q, x.k, x.v, x.w, x.h0, x.dO, x.dhT, cu_seqlens=x.cu, workspace=x.ws),
                  "q k v w h0 dO dhT cu ws"),
    "attn_fwd": (lambda x: gdn.attn_fwd(x.q, x.k, x.v, cu_q=x.cu, cu_k=x.cu_k, k_len=x.k_len, o=x.o, lse=x.lse,
                                        workspace=x.ws), "q k v cu cu_k k_len o lse ws"),
    "attn_bwd": (lambda x: gdn.attn_bwd(x.q, x.k, x.v, x.o, x.lse, x.dO, cu_q=x.cu, cu_k=x.cu_k, workspace=x.ws),
                 "q k v o lse dO cu cu_k ws"),
}


@pytest.mark.parametrize("call", CALLS)
def test_operands_on_two_devices(at, call):
    f, names = CALLS[call]
    for other in names.split():
        with MODE, pytest.raises(ValueError):
            f(operands(0, other, 1))
    assert not at[1]
    with MODE:
        f(operands(0, None, 0))
    assert at[1] == ["gdn_" + call]


@pytest.mark.parametrize("call", CALLS)
def test_operands_on_a_device_that_is_not_current(at, call):
    at[0] = 1
    with MODE, pytest.raises(ValueError):
        CALLS[call][0](operands(0, None, 0))
    assert not at[1]


@pytest.mark.parametrize("size", [lambda: gdn.decay_workspace_bytes(0, 2, 4321, 4000, 2, 4),
                                  lambda: gdn.attn_workspace_bytes(0, 2, 4321, 9000, 4000, 4, 2)])
def test_sizes_are_the_current_device_s(at, size):
    """The plan behind a size counts the device's SMs."""
    assert size() == 1000
    at[0] = 1
    assert size() == 2000
    at[0] = 0
    assert size() == 1000


def test_a_workspace_in_host_memory(at):
    x = operands(0, None, 0)
    x.ws = torch.empty(1 << 20, dtype=torch.uint8)
    for call in ("decay_fwd", "decay_bwd", "attn_fwd", "attn_bwd"):
        with MODE, pytest.raises(ValueError):
            CALLS[call][0](x)
    with MODE:
        x.ws = torch.empty(2 << 20, dtype=torch.uint8, device="cuda:0")[::2]  # (not one piece of memory)
    with MODE, pytest.raises(ValueError):
        CALLS["attn_fwd"][0](x)
