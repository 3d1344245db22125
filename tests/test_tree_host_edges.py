"""Calls of the rotary operators from Python that are refused before a GPU is needed."""

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def binding():
    from speculative_decoding_verification_16_gb300 import build
    build.build()
    from speculative_decoding_verification_16_gb300 import binding
    return binding


def test_interleaved_without_a_truth_value(binding):
    """A flag that is neither true nor false is a type error, and leaves none behind."""
    x, f = torch.zeros(4, 2, 16), torch.zeros(8, dtype=torch.int64)
    p, s = torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    c = torch.zeros(2, 4, 2, 16)
    for bad in (np.ones(2), torch.ones(2)):
        with pytest.raises(TypeError, match="interleaved"):
            binding.spec_verify_rope(x, p, f, interleaved=bad, out=x)
        with pytest.raises(TypeError, match="interleaved"):
            binding.spec_verify_rope_append(None, x, x, p, f, s, c, c.clone(), interleaved=bad)
    with pytest.raises(ValueError, match="CUDA"):
        binding.spec_verify_rope(x, p, f, interleaved=np.bool_(True), out=x)
