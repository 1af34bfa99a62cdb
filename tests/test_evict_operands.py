"""Operands of the eviction that lie in one another are refused before anything is enqueued (CPU)."""
import ctypes

import pytest

import linear_attention_rnn_gb300 as gdn
from test_paged_host import FAKE, P, strides

ARG, WS = -1, -3


@pytest.fixture(scope="module")
def evict():
    gdn.build()
    L = gdn.lib()

    def call(table=1 << 21, to=None, k_len=1 << 22, new=1 << 23, n=3, wide=20, to_wide=16, st=20, sto=16):
        """WS: accepted but for the workspace, which is left out."""
        ptr = lambda x: None if x is None else P(x)
        return L.gdn_cache_evict(FAKE, FAKE, FAKE, ptr(table), ptr(to), ptr(k_len), ptr(new), n, 400, 64, wide, to_wide, 2, 128, 1000,
                                 10, strides(), strides(), st, sto, None, 0, None)
    return call


def test_lengths_that_overlap(evict):
    """Lengths are read by all blocks while one of them writes."""
    at = 1 << 22
    for shift in (0, 4, 8, -4, -8):
        assert evict(k_len=at, new=at + shift) == ARG
    for shift in (12, -12, 1 << 20):
        assert evict(k_len=at, new=at + shift) == WS
    assert evict(n=1, k_len=at, new=at) == ARG and evict(n=1, k_len=at, new=at + 4) == WS


def test_the_table_as_target_with_other_rows(evict):
    """The table itself as target means in place, row by row; other rows of the same memory are other
    sequences' pages."""
    at = 1 << 21
    assert evict(table=at, to=at, to_wide=20, sto=20) == WS
    assert evict(table=at, to=at, to_wide=16, sto=20) == WS         # the first columns of it
    for sto in (16, 19, 21, 40):
        assert evict(table=at, to=at, to_wide=16, sto=sto) == ARG
    assert evict(n=1, table=at, to=at, to_wide=16, sto=16) == WS    # (one row: no distance between rows)
