"""The example that serves a stack from a paged cache.

Tolerance: as for the other example, 2e-2 of the largest output for each attention layer on the
residual path (the two routes differ by roundings of attention's output alone)."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(gdn_lib):
    spec = importlib.util.spec_from_file_location("paged_serving", os.path.join(ROOT, "examples", "paged_serving.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("layers,lens,page", [(1, (300, 77), 32), (2, (130, 1, 40), 16)])
def test_chunks_and_tokens_give_one_pass(example, layers, lens, page):
    stack, rows, outs, _ = example.serve(lens=lens, page=page, layers=layers)
    ref = stack.whole(torch.cat(rows), list(lens)).float()
    assert float((torch.cat(outs).float() - ref).abs().max() / ref.abs().max()) <= 2e-2 * layers


def test_with_a_budget(example):
    _, _, outs, seqs = example.serve(lens=(200, 90), budget=48, page=16)
    assert all(n <= 48 for n in seqs.keys.values()) and seqs.position == {0: 200, 1: 90}
    assert all(len(seqs.pages[s]) == -(-n // 16) for s, n in seqs.keys.items())
    assert all(bool(torch.isfinite(o).all()) for o in outs)
