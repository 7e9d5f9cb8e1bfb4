"""The feed-forward block takes x and the gradient of y in any layout: the same
bits as from a dense copy."""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from mxfp8_block_scaled_dim0_gb300 import feed_forward

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()


def rnd(*shape):
    return torch.randn(*shape, device="cuda").to(BF)


def step(block, x, loss):
    x = x.detach().requires_grad_()
    y = block(x)
    return y, *torch.autograd.grad(loss(y), [x, *block.parameters()])


def test_layouts():
    torch.manual_seed(2)
    block = feed_forward.FeedForward(96, 128)
    dy, head, long = rnd(64, 96), rnd(1), rnd(64 * 96 + 1)
    inputs = [rnd(96, 64).t(), rnd(128, 96)[::2], rnd(64, 192)[:, 96:], rnd(64 * 96 + 1)[1:].view(64, 96),
              rnd(1, 96).expand(64, 96), rnd(32, 2, 96).transpose(0, 1)]
    losses = [lambda y: (y.reshape(-1, 96) * dy).sum(), lambda y: y.sum(),
              lambda y: (y.reshape(-1, 96).t() * dy.view(96, 64)).sum(),
              lambda y: (torch.cat([head, y.reshape(-1)]) * long).sum()]
    for x in inputs:
        for loss in losses:
            want = step(block, x.clone(memory_format=torch.contiguous_format), loss)
            for a, b in zip(step(block, x, loss), want):
                assert torch.equal(a, b)
