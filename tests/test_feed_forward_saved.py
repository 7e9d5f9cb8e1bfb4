"""Blocks saved whole (torch.save of the module) when they had no choice of operators: run as
they were, on operators of 8 bits apart."""
import io

import pytest
import torch

from mxfp8_block_scaled_dim0_gb300 import feed_forward


def test_a_block_without_the_choice():
    block = feed_forward.FeedForward(64, 96, device="cpu")
    for name in ("fused", "bits", "step"):
        block.__dict__.pop(name)
    file = io.BytesIO()
    torch.save(block, file)
    file.seek(0)
    old = torch.load(file, weights_only=False)
    assert (old.fused, old.bits, old.step) == (False, 8, 32)
    with pytest.raises(ValueError, match="multiple of 32, got 33"):
        old(torch.zeros(33, 64, dtype=torch.bfloat16))
