"""Single-token forms (delta_step, decay_step) against their 64-bit definitions.

Tolerances.  A new column of the state is e^g h + k n with n from a dot product
of 128 terms: at most 130 roundings of 2^-24 against the sum of the products'
sizes, which for unit k is at most sqrt(128) max|h|, so 130 * 2^-24 * 11.4 =
8.8e-5 of the largest value (1e-4 below).  The output is rounded to bf16 (unit
roundoff 2^-8: 8 significant bits) after the same sums (1e-4 of the largest).
"""
import pytest
import torch

from oracle import ops
from conftest import assert_rel

pytestmark = pytest.mark.gpu

S_TOL = 1e-4
O_TOL = 2.0 ** -8 + 2e-4


def _rows(R, Hk, Hv, n, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    unit = lambda *s: torch.nn.functional.normalize(r(*s), dim=-1).bfloat16()
    x = dict(q=unit(R, Hk, 128), k=unit(R, Hk, 128), v=r(R, Hv, 128).bfloat16(),
             g=-torch.nn.functional.softplus(r(R, Hv)), beta=torch.sigmoid(r(R, Hv)),
             state=r(n, Hv, 128, 128), decay=-torch.rand(Hv, generator=gen))
    x["slots"] = torch.randperm(n, generator=gen)[:R].to(torch.int32)
    return x


@pytest.mark.parametrize("R,Hk,Hv,n", [(1, 1, 1, 1), (1, 16, 32, 3), (3, 2, 6, 5), (37, 1, 4, 40), (130, 2, 2, 130)])
@pytest.mark.parametrize("delta", [True, False])
def test_step_matches_definition(gdn_lib, R, Hk, Hv, n, delta):
    x = _rows(R, Hk, Hv, n, seed=R + Hv)
    d = {k: t.cuda() for k, t in x.items()}
    for _ in range(2):  # two tokens: the second reads the first one's state
        if delta:
            o = gdn_lib.delta_step(d["q"], d["k"], d["v"], d["g"], d["beta"], d["state"], d["slots"])
            ro, rs = ops.delta_step(x["q"], x["k"], x["v"], x["g"], x["beta"], x["state"], x["slots"].tolist())
        else:
            o = gdn_lib.decay_step(d["q"], d["k"], d["v"], d["decay"], d["state"], d["slots"])
            ro, rs = ops.decay_step(x["q"], x["k"], x["v"], x["decay"], x["state"], x["slots"].tolist())
        assert_rel(o.float().cpu(), ro, O_TOL, "o")
        assert_rel(d["state"].cpu(), rs, S_TOL, "state")
        x["state"] = d["state"].cpu()


def test_rows_without_a_state(gdn_lib):
    x = _rows(6, 2, 4, 8, seed=1)
    x["slots"] = torch.tensor([3, -1, 0, 8, 1 << 30, 5], dtype=torch.int32)  # 8 and beyond: out of range
    d = {k: t.cuda() for k, t in x.items()}
    o = torch.full((6, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    gdn_lib.delta_step(d["q"], d["k"], d["v"], d["g"], d["beta"], d["state"], d["slots"], o=o)
    inside = [s if 0 <= s < 8 else -1 for s in x["slots"].tolist()]
    ro, rs = ops.delta_step(x["q"], x["k"], x["v"], x["g"], x["beta"], x["state"], inside)
    assert torch.equal(o[[1, 3, 4]], torch.zeros_like(o[[1, 3, 4]]))
    assert_rel(o.float().cpu(), ro, O_TOL, "o")
    assert_rel(d["state"].cpu(), rs, S_TOL, "state")
    untouched = [1, 2, 4, 6, 7]
    assert torch.equal(d["state"][untouched].cpu(), x["state"][untouched])


def test_parts_of_one_buffer_and_another_stream(gdn_lib):
    R, Hk, Hv = 9, 2, 4
    x = _rows(R, Hk, Hv, R, seed=2)
    qkv = torch.cat([x["q"].flatten(1), x["k"].flatten(1), x["v"].flatten(1)], 1).cuda()
    q, k, v = qkv.split([Hk * 128, Hk * 128, Hv * 128], 1)
    q, k, v = q.view(R, Hk, 128), k.view(R, Hk, 128), v.view(R, Hv, 128)
    state = x["state"].cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = gdn_lib.decay_step(q, k, v, x["decay"].cuda(), state)
    side.synchronize()
    ro, rs = ops.decay_step(x["q"], x["k"], x["v"], x["decay"], x["state"], range(R))
    assert_rel(o.float().cpu(), ro, O_TOL, "o")
    assert_rel(state.cpu(), rs, S_TOL, "state")


def test_step_continues_the_chunked_forms(gdn_lib):
    """Token T from the step equals token T of a prompt one token longer."""
    from linear_attention_rnn_gb300.inputs import WORKLOADS, make_host
    d = make_host(WORKLOADS["tiny_t1024"].replace(T=261, Hk=2, Hv=4, h0_std=0.1)).to("cuda")
    cut = lambda t: t[:, :260].contiguous()
    _, h = gdn_lib.chunk_fwd(cut(d.q), cut(d.k), cut(d.v), cut(d.g), cut(d.beta), d.h0)
    full, hT = gdn_lib.chunk_fwd(d.q, d.k, d.v, d.g, d.beta, d.h0)
    o = gdn_lib.delta_step(d.q[:, 260], d.k[:, 260], d.v[:, 260], d.g[:, 260].contiguous(),
                           d.beta[:, 260].contiguous(), h)
    assert_rel(o.float().cpu(), full[:, 260].float().cpu(), 2e-2, "o")     # the chunked forward's tolerance
    assert_rel(h.cpu(), hT.cpu(), 1e-2, "state")
    w = -torch.rand(4, device="cuda")
    _, h = gdn_lib.decay_fwd(cut(d.q), cut(d.k), cut(d.v), w, d.h0)
    full, hT = gdn_lib.decay_fwd(d.q, d.k, d.v, w, d.h0)
    o = gdn_lib.decay_step(d.q[:, 260], d.k[:, 260], d.v[:, 260], w, h)
    assert_rel(o.float().cpu(), full[:, 260].float().cpu(), 2e-2, "o (decay)")
    assert_rel(h.cpu(), hT.cpu(), 1e-4, "state (decay)")
