"""The example that runs the mixers together: prompts, then tokens one by one.

Tolerance: the decoded and the whole-prompt outputs go through the same bf16
projections and mixers, whose own tolerances are 2e-2 of the largest value (the
chunked forward's parity tolerance); three mixers add up on the residual path.
"""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(gdn_lib):
    spec = importlib.util.spec_from_file_location("hybrid_stack", os.path.join(ROOT, "examples", "hybrid_stack.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("kinds", [("delta",), ("decay",), ("attn",), ("delta", "decay", "attn")])
def test_tokens_continue_prompts(example, kinds):
    assert example.decode((300, 1, 130), 5, kinds=kinds) <= 2e-2 * len(kinds)


def test_training_pass(example):
    for mixer in example.gradients((200, 1, 77)):
        for t in mixer:
            assert bool(torch.isfinite(t).all())
