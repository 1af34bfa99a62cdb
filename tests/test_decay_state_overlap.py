"""Refusals of decayed linear attention's states that overlap in part -- no GPU needed."""
import ctypes

import pytest

import linear_attention_rnn_gb300 as gdn

P = ctypes.c_void_p
BASE = 1 << 20             # aligned, never dereferenced (validation fails first)
STATE = 4 * 128 * 128 * 4  # one sequence's states of 4 heads
ARG = -1


@pytest.fixture(scope="module")
def L():
    gdn.build()
    return gdn.lib()


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("by", [16, STATE // 2, STATE - 16])
@pytest.mark.parametrize("total", [0, 300])
def test_states_that_overlap_in_part(L, n, by, total):
    x, f = P(BASE), P(BASE << 8)
    for shift in (by, -by, n * STATE - 16):
        y = P(BASE + shift)
        assert L.gdn_decay_fwd(f, f, f, f, x, f, f, y, n, total, 300, 2, 4, 128, 128, 256, 256, 512, f, 1 << 40, None) == ARG
        for h0, dhT in ((None, x), (x, None)):
            assert L.gdn_decay_bwd(f, f, f, f, h0, f, dhT, f, f, f, f, y, n, total, 300, 2, 4, 128, 128, 256, 256, 512, f,
                                   1 << 40, None) == ARG
    # the gradient of the entering state over that state, which the passes read throughout
    assert L.gdn_decay_bwd(f, f, f, f, x, f, None, f, f, f, f, x, n, total, 300, 2, 4, 128, 128, 256, 256, 512, f, 1 << 40,
                           None) == ARG
