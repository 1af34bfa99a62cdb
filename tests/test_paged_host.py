"""Refusals of the head norms with rotation and of the paged cache's operators, devices of their
operands, and their 64-bit definitions against closed forms and differences -- no GPU needed."""
import ctypes
import math
import types

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import linear_attention_rnn_gb300 as gdn
import paged
from oracle import ops

P = ctypes.c_void_p
FAKE = P(1 << 20)          # aligned, never dereferenced (validation fails first)
MISAL = P((1 << 20) + 2)
OK, ARG, SHAPE, WS = 0, -1, -2, -3


@pytest.fixture(scope="module")
def L():
    gdn.build()
    return gdn.lib()


def strides(page=64 * 256, row=256, head=128):
    return ctypes.byref(gdn._PageStrides(page, row, head))


# ---- refusals ---------------------------------------------------------------------------
def test_rope_argument_errors(L):
    def fwd(q=FAKE, k=FAKE, wq=FAKE, pos=FAKE, freq=FAKE, axis=None, qo=FAKE, ko=FAKE, n=4, Hq=4, Hk=2, d=128, axes=1, pairs=64,
            eps=1e-6, sq=512, sk=256, so=512, sko=256):
        return L.gdn_rope_fwd(q, k, wq, None, pos, freq, axis, qo, ko, n, Hq, Hk, d, axes, pairs, 0, eps, sq, sk, so, sko, None)
    assert fwd(n=0) == OK and fwd(n=0, q=None, pos=None) == OK
    assert fwd(d=64) == SHAPE and fwd(pairs=60) == SHAPE and fwd(pairs=72) == SHAPE and fwd(pairs=-8) == SHAPE
    assert fwd(n=-1) == ARG and fwd(Hq=0, sq=0) == ARG and fwd(Hk=-1) == ARG and fwd(axes=0) == ARG
    for eps in (-1e-6, float("nan"), float("inf")):
        assert fwd(eps=eps) == ARG
    assert fwd(q=None) == ARG and fwd(k=None) == ARG and fwd(qo=None) == ARG and fwd(pos=None) == ARG and fwd(freq=None) == ARG
    assert fwd(q=MISAL) == ARG and fwd(wq=MISAL) == ARG and fwd(pos=MISAL) == ARG and fwd(ko=MISAL) == ARG
    assert fwd(sq=256) == ARG and fwd(sk=260) == ARG and fwd(so=256) == ARG and fwd(sko=128) == ARG
    assert fwd(axes=3) == ARG and fwd(axes=2, axis=bytes([2] * 64)) == ARG and fwd(axes=1, axis=bytes([0] * 63 + [1])) == ARG
    assert fwd(n=1 << 29, Hq=4) == ARG

    need = gdn.rope_workspace_bytes(1000, 4, 2)
    assert 0 < gdn.rope_workspace_bytes(1, 4, 2) < need and gdn.rope_workspace_bytes(10, 4, 2, d=64) == 0

    def bwd(q=FAKE, wq=FAKE, dqo=FAKE, dq=FAKE, dwq=FAKE, dwk=None, n=1000, sg=512, so=512, ws=FAKE, nbytes=1 << 30):
        return L.gdn_rope_bwd(q, FAKE, wq, None, FAKE, FAKE, None, dqo, FAKE, dq, FAKE, dwq, dwk, n, 4, 2, 128, 1, 64, 0, 1e-6,
                              512, 256, sg, 256, so, 256, ws, nbytes, None)
    assert bwd(wq=None) == ARG                    # a gradient of a weight that is not there
    assert bwd(dwk=FAKE) == ARG
    assert bwd(q=None) == ARG and bwd(dqo=None) == ARG and bwd(dq=None) == ARG and bwd(dwq=MISAL) == ARG
    assert bwd(sg=256) == ARG and bwd(so=516) == ARG
    assert bwd(nbytes=need - 1) == WS and bwd(ws=None) == WS

    def app(v=FAKE, kp=FAKE, slots=FAKE, n=4, pages=8, page=64, ks=strides(), vs=strides(), sv=256):
        return L.gdn_rope_append(FAKE, FAKE, v, None, None, FAKE, FAKE, None, FAKE, kp, FAKE, slots, n, pages, page, 4, 2, 128,
                                 1, 64, 0, 1e-6, 512, 256, sv, 512, ks, vs, None)
    assert app(n=0) == OK
    assert app(page=8) == SHAPE and app(page=0) == ARG and app(pages=-1) == ARG and app(pages=1 << 26, page=64) == ARG
    assert app(v=None) == ARG and app(kp=None) == ARG and app(slots=None) == ARG and app(slots=MISAL) == ARG and app(sv=128) == ARG
    for bad in (None, strides(row=64), strides(head=132), strides(page=0)):
        assert app(ks=bad) == ARG and app(vs=bad) == ARG


def test_paged_argument_errors(L):
    need = gdn.attn_paged_workspace_bytes(2, 2, 313 * 64, 0, 10000, 4, 2)
    assert need > gdn.attn_paged_workspace_bytes(1, 1, 313 * 64, 0, 100, 4, 2) > 0
    assert gdn.attn_paged_workspace_bytes(1, 1, 64, 0, 64, 4, 2, d=64) == 0

    def fwd(q=FAKE, kp=FAKE, table=FAKE, klen=FAKE, cu=FAKE, o=FAKE, lse=None, n=2, nq=2, mq=0, most=10000, pages=400, page=64, wide=313,
            Hq=4, Hk=2, d=128, scale=0.1, sq=512, ks=strides(), vs=strides(), st=313, ws=FAKE, nbytes=1 << 40):
        return L.gdn_attn_paged(q, kp, FAKE, table, klen, cu, o, lse, n, nq, mq, most, pages, page, wide, Hq, Hk, d, scale, sq, ks, vs,
                                st, ws, nbytes, None)
    assert fwd(n=0) == OK and fwd(nq=0) == OK
    assert fwd(d=64) == SHAPE and fwd(page=40) == SHAPE and fwd(Hq=258, Hk=2, sq=258 * 128) == SHAPE
    assert fwd(Hk=3) == ARG and fwd(nq=-1) == ARG and fwd(most=-1) == ARG and fwd(mq=-1) == ARG
    assert fwd(pages=-1) == ARG and fwd(wide=-1) == ARG
    assert fwd(st=312) == ARG and fwd(wide=1 << 25, st=1 << 25) == ARG
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert fwd(scale=scale) == ARG
    assert fwd(q=None) == ARG and fwd(kp=None) == ARG and fwd(o=None) == ARG and fwd(table=None) == ARG and fwd(klen=None) == ARG
    assert fwd(q=MISAL) == ARG and fwd(table=MISAL) == ARG and fwd(klen=MISAL) == ARG and fwd(lse=MISAL) == ARG and fwd(cu=MISAL) == ARG
    assert fwd(sq=256) == ARG and fwd(cu=None, nq=3) == ARG
    for bad in (None, strides(row=64), strides(head=132)):
        assert fwd(ks=bad) == ARG and fwd(vs=bad) == ARG
    assert fwd(nbytes=need - 1) == WS and fwd(ws=None) == WS

    def weigh(q=FAKE, kp=FAKE, lse=FAKE, table=FAKE, klen=FAKE, w=FAKE, n=2, nq=2, mq=0, pages=400, page=64, wide=313, Hk=2, d=128,
              scale=0.1, sq=512, ks=strides(), st=313, ws=FAKE, nbytes=256):
        return L.gdn_attn_paged_weights(q, kp, lse, table, klen, FAKE, w, n, nq, mq, 10000, pages, page, wide, 4, Hk, d, scale, sq, ks,
                                        st, ws, nbytes, None)
    assert weigh(n=0) == OK and weigh(nq=0) == OK and weigh(pages=0) == OK and weigh(wide=0) == OK
    assert weigh(d=64) == SHAPE and weigh(page=24) == SHAPE and weigh(Hk=3) == ARG and weigh(st=312) == ARG
    assert weigh(lse=None) == ARG and weigh(w=None) == ARG and weigh(table=None) == ARG and weigh(q=None) == ARG
    assert weigh(lse=MISAL) == ARG and weigh(w=MISAL) == ARG and weigh(kp=MISAL) == ARG and weigh(ks=strides(row=64)) == ARG
    assert weigh(scale=-1.0) == ARG and weigh(mq=-1) == ARG and weigh(nbytes=255) == WS

    keep = gdn.cache_evict_workspace_bytes(2, 313 * 64, 1000, 2)
    assert keep >= 2 * 2 * 1000 * 4 and gdn.cache_evict_workspace_bytes(2, 100, 1000, 2) < keep

    def evict(kp=FAKE, w=FAKE, table=FAKE, to=None, klen=FAKE, new=P(1 << 22), n=2, pages=400, page=64, wide=313, to_wide=16, Hk=2, d=128,
              budget=1000, recent=10, vs=strides(), st=313, sto=16, ws=FAKE, nbytes=1 << 30):
        return L.gdn_cache_evict(kp, FAKE, w, table, to, klen, new, n, pages, page, wide, to_wide, Hk, d, budget, recent, strides(),
                                 vs, st, sto, ws, nbytes, None)
    assert evict(n=0) == OK
    assert evict(d=96) == SHAPE and evict(page=17) == SHAPE
    assert evict(Hk=0) == ARG and evict(budget=-1) == ARG and evict(recent=-1) == ARG and evict(wide=-1) == ARG and evict(st=1) == ARG
    assert evict(kp=None) == ARG and evict(w=None) == ARG and evict(table=None) == ARG and evict(klen=None) == ARG
    assert evict(klen=P(1 << 21), new=P(1 << 21)) == ARG     # lengths read and written at once
    assert evict(new=None) == ARG and evict(new=MISAL) == ARG and evict(to=MISAL) == ARG and evict(vs=None) == ARG
    # target pages for fewer keys than may stay
    assert evict(to=P(1 << 21), to_wide=15) == ARG and evict(to=P(1 << 21), sto=15) == ARG
    assert evict(nbytes=keep - 1 - 255) == WS and evict(ws=None) == WS


def test_bindings_validate_before_calling():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    i, f = torch.zeros(4, dtype=torch.int32), torch.zeros(64)
    pages, table = torch.zeros(3, 16, 2, 128, dtype=torch.bfloat16), torch.zeros(4, 1, dtype=torch.int32)
    for call in (lambda: gdn.rope_fwd(x, x, i, f), lambda: gdn.rope_bwd(x, x, i, f, x, x),
                 lambda: gdn.rope_append(x, x, x, i, f, pages, pages, i), lambda: gdn.attn_paged(x, pages, pages, table, i, cu_q=i),
                 lambda: gdn.attn_paged_weights(x, pages, f, table, i, f, cu_q=i),
                 lambda: gdn.cache_evict(pages, pages, f, table, i, 4)):
        with pytest.raises(ValueError):    # CPU tensors
            call()


# ---- operands of the bindings: shapes on devices that are not there, a stand-in library --------
MODE = FakeTensorMode(allow_non_fake_inputs=True)
BF, F, I = torch.bfloat16, torch.float32, torch.int32
NAMES = ("rope_fwd", "rope_bwd", "rope_append", "attn_paged", "attn_paged_weights", "cache_evict")


@pytest.fixture
def calls(monkeypatch):
    calls = []

    def stand_in(name):
        def f(*args):
            if name.endswith("workspace_bytes"):
                return 1000
            calls.append(name)
            return 0
        return f
    sizes = ["gdn_rope_workspace_bytes", "gdn_attn_paged_workspace_bytes", "gdn_cache_evict_workspace_bytes"]
    monkeypatch.setattr(gdn, "lib", lambda: types.SimpleNamespace(**{n: stand_in(n) for n in ["gdn_" + n for n in NAMES] + sizes}))
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(gdn, "_several_devices", True, raising=False)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    gdn._planned_bytes.cache_clear()
    yield calls
    gdn._planned_bytes.cache_clear()


def operands(other=None, **change):
    shapes = dict(q=(4, 2, 128, BF), k=(4, 1, 128, BF), v=(4, 1, 128, BF), pos=(4, I), freq=(64, F), wq=(128, F), wk=(128, F),
                  q_out=(4, 2, 128, BF), k_out=(4, 1, 128, BF), gq=(4, 2, 128, BF), gk=(4, 1, 128, BF), kp=(3, 16, 1, 128, BF),
                  vp=(3, 16, 1, 128, BF), slots=(4, I), table=(2, 5, I), to=(2, 5, I), k_len=(2, I), cu=(3, I), o=(4, 2, 128, BF),
                  lse=(4, 2, F), weights=(3, 1, 16, F), new_len=(2, I), ws=(1 << 16, torch.uint8))
    shapes.update(change)
    with MODE:
        return types.SimpleNamespace(**{n: torch.empty(s[:-1], dtype=s[-1], device=f"cuda:{int(n == other)}")
                                        for n, s in shapes.items()})


CALLS = {
    "rope_fwd": (lambda x: gdn.rope_fwd(x.q, x.k, x.pos, x.freq, q_weight=x.wq, k_weight=x.wk, q_out=x.q_out, k_out=x.k_out),
                 "q k pos freq wq wk q_out k_out"),
    "rope_bwd": (lambda x: gdn.rope_bwd(x.q, x.k, x.pos, x.freq, x.gq, x.gk, q_weight=x.wq, k_weight=x.wk, dq=x.q_out, dk=x.k_out,
                                        workspace=x.ws), "q k pos freq gq gk wq wk q_out k_out ws"),
    "rope_append": (lambda x: gdn.rope_append(x.q, x.k, x.v, x.pos, x.freq, x.kp, x.vp, x.slots, q_weight=x.wq, k_weight=x.wk,
                                              q_out=x.q_out), "q k v pos freq kp vp slots wq wk q_out"),
    "attn_paged": (lambda x: gdn.attn_paged(x.q, x.kp, x.vp, x.table, x.k_len, cu_q=x.cu, o=x.o, lse=x.lse, workspace=x.ws),
                   "q kp vp table k_len cu o lse ws"),
    "attn_paged_weights": (lambda x: gdn.attn_paged_weights(x.q, x.kp, x.lse, x.table, x.k_len, x.weights, cu_q=x.cu, workspace=x.ws),
                           "q kp lse table k_len weights cu ws"),
    "cache_evict": (lambda x: gdn.cache_evict(x.kp, x.vp, x.weights, x.table, x.k_len, 9, to_table=x.to, new_len=x.new_len,
                                              workspace=x.ws), "kp vp weights table k_len to new_len ws"),
}


@pytest.mark.parametrize("call", CALLS)
def test_operands_on_two_devices(calls, call):
    f, names = CALLS[call]
    for other in names.split():
        with MODE, pytest.raises(ValueError):
            f(operands(other))
    assert not calls
    with MODE:
        f(operands())
    assert calls == ["gdn_" + call]


@pytest.mark.parametrize("call,change", [
    ("rope_fwd", dict(k=(5, 1, 128, BF))), ("rope_fwd", dict(pos=(5, I))), ("rope_fwd", dict(pos=(2, 5, I))), ("rope_fwd", dict(pos=(4, F))),
    ("rope_fwd", dict(freq=(64, torch.float64))), ("rope_fwd", dict(wq=(64, F))), ("rope_fwd", dict(q_out=(4, 1, 128, BF))),
    ("rope_fwd", dict(q=(4, 2, 128, torch.float16))), ("rope_bwd", dict(gq=(4, 1, 128, BF))), ("rope_bwd", dict(gk=(3, 1, 128, BF))),
    ("rope_append", dict(v=(4, 2, 128, BF))), ("rope_append", dict(kp=(3, 16, 2, 128, BF))), ("rope_append", dict(vp=(4, 16, 1, 128, BF))),
    ("rope_append", dict(slots=(3, I))), ("rope_append", dict(slots=(4, torch.int64))),
    ("attn_paged", dict(table=(3, 5, I))), ("attn_paged", dict(table=(2, 5, torch.int64))), ("attn_paged", dict(k_len=(3, I))),
    ("attn_paged", dict(kp=(3, 16, 1, 64, BF))), ("attn_paged", dict(vp=(3, 32, 1, 128, BF))), ("attn_paged", dict(o=(4, 1, 128, BF))),
    ("attn_paged", dict(ws=(100, torch.uint8))), ("attn_paged_weights", dict(lse=(4, 1, F))),
    ("attn_paged_weights", dict(weights=(3, 16, 1, F))), ("cache_evict", dict(weights=(3, 16, 1, F))), ("cache_evict", dict(to=(3, 5, I))),
    ("cache_evict", dict(new_len=(3, I))), ("cache_evict", dict(k_len=(2, torch.int64))), ("cache_evict", dict(ws=(100, torch.uint8))),
])
def test_shapes_and_types(calls, call, change):
    with MODE, pytest.raises(ValueError):
        CALLS[call][0](operands(**change))
    assert not calls


def test_axes_of_pairs(calls):
    x = operands(pos=(3, 4, I))
    with MODE:
        gdn.rope_fwd(x.q, x.k, x.pos, x.freq, pair_axis=[0] * 16 + [1] * 24 + [2] * 24)
    for bad in ([0] * 63, [0] * 63 + [-1], [0] * 63 + [256]):
        with MODE, pytest.raises(ValueError):
            gdn.rope_fwd(x.q, x.k, x.pos, x.freq, pair_axis=bad)
    with MODE, pytest.raises(ValueError):
        gdn.rope_fwd(x.q, x.k, None, x.freq)
    assert calls == ["gdn_rope_fwd"]


# ---- the definitions: closed forms and differences ----------------------------------------
def r64(*shape, seed):
    return torch.from_numpy(np.random.default_rng([seed, *shape]).standard_normal(shape))


def difference(f, x, dx, eps=1e-6):
    return float((f(x + eps * dx) - f(x - eps * dx)) / (2 * eps))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_gradients_against_differences(interleaved, norm):
    x, w, dy = r64(5, 3, 16, seed=1), r64(16, seed=2) if norm else None, r64(5, 3, 16, seed=3)
    angle = ops.angles(torch.arange(10).view(2, 5), torch.tensor([0.1, 0.7, 1.3, 2.0, 0.4, 0.0]), (0, 1, 1, 0, 0, 1))
    loss = lambda x, w: (ops.rope(x, w, angle, interleaved, 1e-2)[0] * dy).sum()
    dx, _, dw, _ = ops.rope_bwd(x, w, angle, interleaved, 1e-2, dy)
    a, b = r64(5, 3, 16, seed=4), r64(16, seed=5)
    assert difference(lambda t: loss(t, w), x, a) == pytest.approx(float((dx * a).sum()), rel=1e-6)
    if norm:
        assert difference(lambda t: loss(x, t), w, b) == pytest.approx(float((dw * b).sum()), rel=1e-6)


def test_rope_closed_forms():
    x = r64(3, 2, 8, seed=1)
    half = ops.angles(torch.tensor([0, 1, 2]), torch.full((4,), math.pi))
    y, _ = ops.rope(x, None, half, False, 0.0)        # half a turn, a whole one
    assert torch.allclose(y, x * torch.tensor([1.0, -1.0, 1.0]).double()[:, None, None], atol=1e-6)
    # scores of turned rows depend on the distance of their positions alone
    freq = torch.tensor([0.3, 0.05, 1.0, 0.7])
    at = lambda t, x, i: ops.rope(x[None, None], None, ops.angles(torch.tensor([t]), freq), i, 0.0)[0][0, 0]
    for i in (False, True):
        assert float(at(7, x[0, 0], i) @ at(4, x[1, 1], i)) == pytest.approx(float(at(103, x[0, 0], i) @ at(100, x[1, 1], i)))
    n, _ = ops.rope(x, torch.ones(8), 0 * half, False, 0.0)
    assert torch.allclose(n.square().mean(-1), torch.ones(3, 2).double())


def test_paged_definitions():
    """Pages give what the same keys in one piece give; weights add up to the queries; eviction by hand."""
    ql, kl = [3, 5], [40, 5]
    x = paged.cache(ql, kl, 4, 2, 16, seed=1, nan=False)
    r = ops.attn_paged(x["q"], x["kp"], x["vp"], x["table"], ql, kl, 0.1)
    flat = lambda p: torch.cat([p.reshape(-1, 2, 128)[ops.rows_of(x["table"][s], m, 16, p.shape[0])] for s, m in enumerate(kl)])
    one = ops.attn(x["q"], flat(x["kp"]), flat(x["vp"]), ql, [0, 40], kl, 0.1)
    assert torch.allclose(r["o"], one["o"]) and torch.allclose(r["lse"], one["lse"])
    w, _ = ops.attn_paged_weights(x["q"], x["kp"], r["lse"], x["table"], ql, kl, torch.zeros_like(x["weights"]), 0.1)
    assert float(w.sum()) == pytest.approx(8 * 4)
    k = torch.arange(16.0).view(1, 16, 1, 1).expand(1, 16, 1, 128)
    weight = torch.tensor([5.0, 1, 9, 9, 2, float("nan"), 0, 7] + [100.0] * 8).view(1, 1, 16)
    t = torch.tensor([[0]])
    nk, _, nw, n = ops.cache_evict(k, k, weight, t, [8], 5, 2, t)   # 6 and 7 are the last ones; 2, 3, 0 the heaviest others
    assert n == [5] and nk[0, :5, 0, 0].tolist() == [0, 2, 3, 6, 7] and nk[0, 5:, 0, 0].tolist() == list(range(5, 16))
    assert nw[0, 0, :5].tolist() == [5, 9, 9, 0, 7]
