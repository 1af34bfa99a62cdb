"""Refusals of the operators around the chunked rule, and their 64-bit definitions
against differences -- no GPU needed."""
import ctypes

import numpy as np
import pytest
import torch

import linear_attention_rnn_gb300 as gdn
from oracle import ops

P = ctypes.c_void_p
FAKE = P(1 << 20)          # aligned, never dereferenced (validation fails first)
MISAL = P((1 << 20) + 2)
OK, ARG, SHAPE, WS = 0, -1, -2, -3


@pytest.fixture(scope="module")
def L():
    gdn.build()
    return gdn.lib()


# ---- refusals ---------------------------------------------------------------------------
def test_step_argument_errors(L):
    def delta(q=FAKE, beta=FAKE, state=FAKE, slots=FAKE, o=FAKE, R=4, n=4, Hk=2, Hv=4, d=128, sq=256, sv=512):
        return L.gdn_delta_step(q, FAKE, FAKE, FAKE, beta, state, slots, o, R, n, Hk, Hv, d, d, sq, 256, sv, None)

    def decay(w=FAKE, R=4, Hk=2, Hv=4, d=128, sk=256):
        return L.gdn_decay_step(FAKE, FAKE, FAKE, w, FAKE, None, FAKE, R, 4, Hk, Hv, d, d, 256, sk, 512, None)
    assert delta(R=0) == OK and decay(R=0) == OK   # nothing to do
    assert delta(d=64) == SHAPE and decay(d=64) == SHAPE
    assert delta(R=-1) == ARG and delta(n=-1) == ARG
    assert delta(Hk=3) == ARG and decay(Hk=0) == ARG
    assert delta(q=None) == ARG and delta(beta=None) == ARG and delta(state=None) == ARG and delta(o=None) == ARG
    assert decay(w=None) == ARG
    assert delta(q=MISAL) == ARG and delta(slots=MISAL) == ARG
    assert delta(sq=128) == ARG        # rows that overlap
    assert delta(sv=516) == ARG        # rows off 16 bytes
    assert decay(sk=260) == ARG
    assert delta(R=1 << 28, Hv=4) == ARG


def test_decay_argument_errors(L):
    small = gdn.decay_workspace_bytes(0, 2, 300, 200, 2, 4)
    need_b = gdn.decay_workspace_bytes(1, 2, 300, 200, 2, 4)
    assert 0 < small < need_b          # the backward keeps running sums of the shared heads
    assert gdn.decay_workspace_bytes(0, 2, 300, 200, 2, 4, dk=64) == 0
    assert gdn.decay_workspace_bytes(0, 2, 300, 200, 3, 4) == 0

    need = gdn.decay_workspace_bytes(0, 1, 20000, 20000, 2, 4)  # one long sequence: states of its segments

    def fwd(q=FAKE, w=FAKE, cu=FAKE, o=FAKE, h0=None, n=1, total=20000, most=20000, Hk=2, Hv=4, d=128, sq=256, ws=FAKE,
            nbytes=1 << 40):
        return L.gdn_decay_fwd(q, FAKE, FAKE, w, h0, cu, o, None, n, total, most, Hk, Hv, d, d, sq, 256, 512, ws, nbytes,
                               None)
    assert fwd(n=0) == OK and fwd(total=0) == OK
    assert fwd(d=96) == SHAPE
    assert fwd(n=-1) == ARG and fwd(total=-1) == ARG and fwd(most=-1) == ARG and fwd(Hk=3) == ARG
    assert fwd(q=None) == ARG and fwd(w=None) == ARG and fwd(o=None) == ARG
    assert fwd(q=MISAL) == ARG and fwd(h0=MISAL) == ARG and fwd(cu=MISAL) == ARG
    assert fwd(sq=128) == ARG and fwd(sq=260) == ARG
    assert fwd(cu=None, n=3) == ARG          # equal lengths
    assert fwd(nbytes=need - 1) == WS and fwd(ws=None) == WS

    def bwd(dO=FAKE, dv=FAKE, nbytes=1 << 40):
        return L.gdn_decay_bwd(FAKE, FAKE, FAKE, FAKE, None, dO, None, FAKE, FAKE, FAKE, dv, None, 2, 300, 200, 2, 4,
                               128, 128, 256, 256, 512, FAKE, nbytes, None)
    assert bwd(dO=None) == ARG and bwd(dv=None) == ARG and bwd(dv=MISAL) == ARG
    assert bwd(nbytes=need_b - 1) == WS


def test_attn_argument_errors(L):
    need = gdn.attn_workspace_bytes(0, 2, 2, 20000, 10000, 4, 2)
    assert need > gdn.attn_workspace_bytes(0, 2, 2, 20000, 128, 4, 2) > 0  # splits of long contexts
    assert gdn.attn_workspace_bytes(0, 1, 128, 128, 128, 4, 3) == 0
    assert gdn.attn_workspace_bytes(0, 1, 128, 128, 128, 4, 2, d=64) == 0

    def fwd(q=FAKE, k=FAKE, cu_q=FAKE, klen=None, o=FAKE, lse=None, n=2, nq=2, nk=20000, most=10000, Hq=4, Hk=2, d=128,
            scale=0.1, sq=512, ws=FAKE, nbytes=1 << 40):
        return L.gdn_attn_fwd(q, k, FAKE, cu_q, FAKE, klen, o, lse, n, nq, nk, most, Hq, Hk, d, scale, sq, 256, 256, ws,
                              nbytes, None)
    assert fwd(n=0) == OK and fwd(nq=0) == OK
    assert fwd(d=64) == SHAPE and fwd(Hq=258, Hk=2, sq=258 * 128) == SHAPE   # 129 heads to a key head
    assert fwd(Hk=3) == ARG and fwd(nq=-1) == ARG and fwd(most=-1) == ARG
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert fwd(scale=scale) == ARG
    assert fwd(q=None) == ARG and fwd(k=None) == ARG and fwd(o=None) == ARG
    assert fwd(q=MISAL) == ARG and fwd(cu_q=MISAL) == ARG and fwd(klen=MISAL) == ARG and fwd(lse=MISAL) == ARG
    assert fwd(sq=256) == ARG
    assert fwd(cu_q=None, nq=3) == ARG
    assert fwd(nbytes=need - 1) == WS and fwd(ws=None) == WS

    def bwd(lse=FAKE, dO=FAKE, dk=FAKE, nbytes=1 << 40):
        return L.gdn_attn_bwd(FAKE, FAKE, FAKE, FAKE, lse, dO, FAKE, FAKE, FAKE, dk, FAKE, 2, 256, 256, 4, 2, 128, 0.1,
                              512, 256, 256, FAKE, nbytes, None)
    assert bwd(lse=None) == ARG and bwd(dO=None) == ARG and bwd(dk=None) == ARG and bwd(dO=MISAL) == ARG
    assert bwd(nbytes=16) == WS


def test_bindings_validate_before_calling():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # CPU tensors
        gdn.decay_fwd(x, x, x, torch.zeros(2), cu_seqlens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        gdn.attn_fwd(x, x, x, cu_q=torch.zeros(2, dtype=torch.int32), cu_k=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        gdn.delta_step(x, x, x, torch.zeros(4, 2), torch.zeros(4, 2), torch.zeros(4, 2, 128, 128))
    with pytest.raises(ValueError):  # cu_q without cu_k
        gdn.attn_fwd(x, x, x, cu_q=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):  # neither packed nor batched
        gdn.decay_fwd(x, x, x, torch.zeros(2))


# ---- the definitions: closed forms and differences ----------------------------------------
def r64(*shape, seed):
    return torch.from_numpy(np.random.default_rng([seed, *shape]).standard_normal(shape))


def difference(f, x, dx, eps=1e-6):
    return float((f(x + eps * dx) - f(x - eps * dx)) / (2 * eps))


@pytest.mark.parametrize("which", ["q", "k", "v", "h0"])
def test_decay_gradients_against_differences(which):
    lens = [5, 0, 7]
    x = dict(q=r64(12, 1, 6, seed=1), k=r64(12, 1, 6, seed=2), v=r64(12, 2, 6, seed=3), h0=r64(3, 2, 6, 6, seed=4))
    w = torch.tensor([-0.3, -0.05], dtype=torch.float64)
    dO, dhT = r64(12, 2, 6, seed=5), r64(3, 2, 6, 6, seed=6)

    def loss(t):
        y = dict(x, **{which: t})
        o, hT = ops.decay_fwd(y["q"], y["k"], y["v"], w, y["h0"], lens)
        return (o * dO).sum() + (hT * dhT).sum()
    grads = dict(zip(("q", "k", "v", "h0"), ops.decay_bwd(x["q"], x["k"], x["v"], w, x["h0"], dO, dhT, lens)))
    dx = r64(*x[which].shape, seed=7)
    assert difference(loss, x[which], dx) == pytest.approx(float((grads[which] * dx).sum()), rel=1e-6)


@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_attention_gradients_against_differences(which):
    ql, kl, k0 = [4, 3, 2], [6, 3, 1], [0, 6, 9]      # a continued one, a whole one, more queries than keys
    x = dict(q=r64(9, 4, 6, seed=1), k=r64(10, 2, 6, seed=2), v=r64(10, 2, 6, seed=3))
    dO = r64(9, 4, 6, seed=4)

    def loss(t):
        y = dict(x, **{which: t})
        return (ops.attn(y["q"], y["k"], y["v"], ql, k0, kl, 0.4)["o"] * dO).sum()
    g = ops.attn(x["q"], x["k"], x["v"], ql, k0, kl, 0.4, dO)["d" + which]
    dx = r64(*x[which].shape, seed=5)
    assert difference(loss, x[which], dx) == pytest.approx(float((g * dx).sum()), rel=1e-6)


def test_attention_rows_without_keys_and_uniform_rows():
    q, k, v = torch.zeros(3, 1, 4), torch.zeros(2, 1, 4), torch.arange(8.0).reshape(2, 1, 4)
    r = ops.attn(q, k, v, [3], [0], [2], 1.0)
    assert float(r["lse"][0, 0]) == -float("inf") and not r["o"][0].any()     # sees no key
    assert torch.equal(r["o"][1, 0], v[0, 0].double())                         # sees the first one
    assert torch.allclose(r["o"][2, 0], v[:, 0].double().mean(0))              # even weights


def test_steps_are_tokens_of_the_recurrences():
    T, Hv = 6, 2
    q, k, v = r64(T, 1, 8, seed=1), r64(T, 1, 8, seed=2), r64(T, Hv, 8, seed=3)
    w = torch.tensor([-0.2, -1.0], dtype=torch.float64)
    state = torch.zeros(1, Hv, 8, 8, dtype=torch.float64)
    o, hT = ops.decay_fwd(q, k, v, w, None, [T])
    for t in range(T):
        ot, state = ops.decay_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], w, state, [0])
        assert torch.allclose(ot[0], o[t])
    assert torch.allclose(state[0], hT[0])
    # the delta rule with beta = 0 only decays; with beta = 1 and a unit key it stores v under k
    g, zero, one = torch.full((1, Hv), -0.5, dtype=torch.float64), torch.zeros(1, Hv), torch.ones(1, Hv)
    unit = torch.nn.functional.normalize(k[:1], dim=-1)
    _, s0 = ops.delta_step(q[:1], unit, v[:1], g, zero, state, [0])
    assert torch.allclose(s0, np.exp(-0.5) * state)
    _, s1 = ops.delta_step(q[:1], unit, v[:1], g, one, state, [0])
    assert torch.allclose(torch.einsum("i,hij->hj", unit[0, 0], s1[0]), v[0])
