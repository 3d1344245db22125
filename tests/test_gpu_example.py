"""The speculative decoding example: greedy output with drafts is that without."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(cuda_lib):
    spec = importlib.util.spec_from_file_location(
        "speculative_decode", os.path.join(ROOT, "examples", "speculative_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("page,block", [(16, 6), (5, 3)])
def test_greedy_speculation_changes_nothing(example, page, block):
    """fp32: products of one row and of a block differ in their last bits only, far
    below the gap between the two best of 1,009 logits."""
    shape = (1009, 4, 2, 32, 400, page, torch.float32, 3)
    target, draft = example.Toy(*shape), example.Toy(*shape, noise=0.3)
    prompts = [[5, 9], [1] * 40, list(range(100)), [7]]
    kw = dict(page=page, pages=400, width=60)
    spec, drafted, accepted = example.generate(target, draft, prompts, 30, block, **kw)
    plain, _, _ = example.generate(target, draft, prompts, 30, 1, **kw)
    assert spec == plain
    assert 0 < accepted < drafted


def test_sampling_in_bf16_runs(example):
    shape = (5003, 8, 2, 64, 300, 16, torch.bfloat16, 5)
    target, draft = example.Toy(*shape), example.Toy(*shape, noise=0.2)
    out, drafted, accepted = example.generate(target, draft, [[3] * n for n in (1, 17, 64)], 24, 5,
                                              page=16, pages=300, width=16, temperature=0.8)
    assert all(len(o) == 24 for o in out) and 0 < accepted <= drafted
    same, drafted, accepted = example.generate(target, target, [[3] * 9], 24, 5, page=16, pages=300,
                                               width=16, temperature=0.8)
    assert accepted >= 0.9 * drafted  # a drafter that is the target
