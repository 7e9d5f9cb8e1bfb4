"""The feed-forward block against 64 bits of what it computes, its casts included:
the same MX casts (the casts' own tests hold them to the byte) and roundings to
bf16, everything between them in 64 bits.

Tolerance.  What is left are the fp32 errors of the operators (under 2^-18 of a value)
and what they tip over: a rounding to bf16 goes the other way for at most one value
in 2^8, by 2^-8 of it: 2^-12 in the 2-norm.  A cast of such values, and of the fp32
ones, moves by a unit of e4m3 (2^-3) where a value lies within 2^-8 of a boundary, one
tipped value in 2^4: 2^-3 (2^-12)^(1/2) = 2^-9.  n casts on the way, each twice that: n
2^-8 of a result's 2-norm, independent as they are, where the casts themselves move it
by n 2^-4.
"""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
import plain64
from mxfp8_block_scaled_dim0_gb300 import feed_forward

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()


def cast(x):
    """What the casts of bf16 x along its rows and along its columns stand for."""
    q0, s0, q1, s1 = mx.cast_dim0_dim1(x.to(BF).contiguous())
    return plain64.mx_values(q0, s0), plain64.mx_values(q1, s1).t()


def block64(x, nw, nb, w1, w2, eps, dy):
    n, mean, rstd = plain64.layer_norm(x, nw, nb, eps)
    n0, n1 = cast(n)
    a0, a1 = cast(w1)
    b0, b1 = cast(w2)
    gu = (n0 @ a0.t()).to(BF)
    h0, h1 = cast(plain64.swiglu(gu))
    y = x.double() + (h0 @ b0.t()).to(BF).double()
    d0, d1 = cast(dy)
    dw2 = d1.t() @ h1
    dh = (d0 @ b1).to(BF)
    e0, e1 = cast(plain64.swiglu_backward(dh, cast(gu)[0]))
    dw1 = e1.t() @ n1
    dn = (e0 @ a1).to(BF)
    dx, dnw, dnb = plain64.layer_norm_backward(dn, cast(x)[0], nw, mean, rstd)[0]
    return y, (dy.double() + dx.to(BF).double(), dx), dnw, dnb, dw1, dw2


@pytest.mark.parametrize("T,dim,hidden", [(64, 96, 160), (320, 256, 512), (1024, 512, 1024)])
def test_block(T, dim, hidden):
    torch.manual_seed(7)
    block = feed_forward.FeedForward(dim, hidden)
    with torch.no_grad():
        block.norm_w.add_(0.2 * torch.randn_like(block.norm_w))
        block.norm_b.add_(0.2 * torch.randn_like(block.norm_b))
    x = torch.randn(T, dim, device="cuda").to(BF).requires_grad_()
    dy = torch.randn(T, dim, device="cuda").to(BF)
    y = block(x)
    got = torch.autograd.grad(y, [x, block.norm_w, block.norm_b, block.w1, block.w2], dy)
    p = [t.detach() for t in (x, block.norm_w, block.norm_b, block.w1, block.w2)]
    want = block64(*p, block.eps, dy)

    def off(a, b, scale=None):
        return float((a.detach().double() - b).norm() / (b if scale is None else scale).norm())

    assert off(y, want[0]) < 4 * 2.0 ** -8
    # without the identity's share, which no cast touches
    dx, through = want[1]
    assert off(got[0], dx, through) < 8 * 2.0 ** -8 + 2.0 ** -8 * float(dx.norm() / through.norm())
    for a, b, casts in zip(got[1:], want[2:], (8, 8, 7, 4)):
        assert off(a, b) < casts * 2.0 ** -8
