"""How the feed-forward block joins its operators, on the CPU: the operators
replaced by plain 64-bit stand-ins (a cast keeps every bit), so that nothing but
the block's own steps is between its gradients and those of autograd.

Tolerance: both sides add up the same products in 64 bits, in another order:
2^-53 of sums of up to 256 terms, a few operators deep, far below 1e-12 of the
2-norm.
"""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from mxfp8_block_scaled_dim0_gb300 import feed_forward

import plain64


def dense(*ts):
    """What the C entry points ask of a tensor."""
    for t in ts:
        assert t.is_contiguous() and t.data_ptr() % 16 == 0


@pytest.fixture
def block(monkeypatch):
    def cast(x):
        dense(x)
        none = torch.zeros(1)
        return x.clone(), none, x.t().contiguous(), none

    def layer_norm(x, w, b, eps, save):
        dense(x, w, b)
        return (*plain64.layer_norm(x, w, b, eps), x.clone(), torch.zeros(1))

    def layer_norm_backward(dy, saved, w, mean, rstd):
        dense(dy)
        return plain64.layer_norm_backward(dy, saved[0], w, mean, rstd)[0]

    def swiglu(gu, save):
        dense(gu)
        return plain64.swiglu(gu), gu.clone(), torch.zeros(1)

    def swiglu_backward(dh, saved):
        dense(dh)
        return plain64.swiglu_backward(dh, saved[0])

    for name, f in (("cast_dim0_dim1", cast), ("layer_norm", layer_norm),
                    ("layer_norm_backward", layer_norm_backward), ("swiglu", swiglu),
                    ("swiglu_backward", swiglu_backward),
                    ("matmul", lambda qa, sa, qb, sb: qa @ qb.t())):
        monkeypatch.setattr(mx, name, f)
    torch.manual_seed(5)
    block = feed_forward.FeedForward(64, 96, device="cpu").double()
    with torch.no_grad():
        block.norm_w.add_(0.2 * torch.randn_like(block.norm_w))
        block.norm_b.add_(0.2 * torch.randn_like(block.norm_b))
    return block


def plain(block, x):
    y, _, _ = plain64.layer_norm(x, block.norm_w, block.norm_b, block.eps)
    return x + plain64.swiglu(y @ block.w1.t()) @ block.w2.t()


def off(a, b):
    return float((a - b).detach().norm() / b.detach().norm())


def leaves(block, x):
    return [x, block.norm_w, block.norm_b, block.w1, block.w2]


def check(block, x, loss):
    """loss(y) through the block against loss(y) through autograd."""
    x = x.detach().requires_grad_()
    y = block(x)
    got = torch.autograd.grad(loss(y), leaves(block, x))
    y64 = plain(block, x.reshape(-1, x.shape[-1])).reshape(x.shape)
    want = torch.autograd.grad(loss(y64), leaves(block, x))
    assert off(y, y64) < 1e-12
    for a, b in zip(got, want):
        assert off(a, b) < 1e-12


def test_gradients(block):
    dy = torch.randn(64, 64, dtype=torch.float64)
    check(block, torch.randn(64, 64, dtype=torch.float64), lambda y: (y * dy).sum())
    dy = dy.reshape(2, 32, 64)
    check(block, torch.randn(2, 32, 64, dtype=torch.float64), lambda y: (y * dy).sum())


def test_second_derivatives_are_refused(block):
    """The operators leave no graph behind: differentiated again, the block would
    give the derivative of the residual path alone, or none where the gradient of y
    is a constant.  An error, not a number."""
    x = torch.randn(32, 64, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(32, 64, dtype=torch.float64)
    for loss in (lambda y: y.square().sum(), lambda y: (y * dy).sum(), lambda y: y.sum() + x.pow(3).sum()):
        want = torch.autograd.grad(loss(block(x)), leaves(block, x))
        got = torch.autograd.grad(loss(block(x)), leaves(block, x), create_graph=True)
        for a, b in zip(got, want):
            assert torch.equal(a, b) and not b.requires_grad
            with pytest.raises(RuntimeError, match="no second derivative"):
                a.square().sum().backward(retain_graph=True)


def test_inputs_of_any_layout(block):
    """x or the gradient of y transposed, expanded, or off the 16-byte boundary."""
    x = torch.randn(64, 64, dtype=torch.float64)
    shifted = torch.randn(64 * 64 + 1, dtype=torch.float64)[1:].view(64, 64)
    dy = torch.randn(64, 64, dtype=torch.float64)
    for v in (x.t(), x[::2], shifted, x[:1].expand(32, 64)):
        check(block, v, lambda y: (y * dy[:len(v)]).sum())
    check(block, x, lambda y: (y.t() * dy).sum())
    check(block, x, lambda y: y.sum())
    head = torch.randn(1, dtype=torch.float64)
    check(block, x, lambda y: (torch.cat([head, y.reshape(-1)]) * torch.arange(4097)).sum())
