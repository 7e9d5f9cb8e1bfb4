"""The feed-forward block by the joined products, and a chain of the 4-bit operators as a
server runs it: equal, bit for bit, to the operators called one after another, which their
own tests hold to 64 bits; in 8 bits also against the unquantised block; captured into a
graph; on another stream.

Tolerance in 8 bits: as in test_gpu_feed_forward.py, n casts within n 2^-4 of the 2-norm.
"""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from mxfp8_block_scaled_dim0_gb300 import feed_forward
from test_gpu_feed_forward import reference

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()
    yield
    torch.cuda.synchronize()
    assert mx.mx_watchdog(clear=True) == 0


def rnd(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(BF)


def block_of(dim, hidden, bits, seed=3):
    torch.manual_seed(seed)
    block = feed_forward.FeedForward(dim, hidden, fused=True, bits=bits)
    with torch.no_grad():
        block.norm_w.add_(0.2 * torch.randn_like(block.norm_w))
        block.norm_b.add_(0.2 * torch.randn_like(block.norm_b))
    return block


def by_hand(block, x, dy):
    """y and the gradients, an operator at a time."""
    d0, d1, product = ((mx.cast_dim0, mx.cast_dim1, mx.matmul) if block.bits == 8 else
                       (mx.cast_fp4_dim0, mx.cast_fp4_dim1, mx.matmul_fp4))
    w1, w2, F = block.w1.detach(), block.w2.detach(), block.w2.shape[1]
    n, mean, rstd, xq, xs = mx.layer_norm(x, block.norm_w, block.norm_b, block.eps, save=True)
    gate, up = d0(w1[:F].contiguous()), d0(w1[F:].contiguous())
    h, q, s = mx.matmul_swiglu(*d0(n), *zip(gate, up), save=True, bits=block.bits)
    y = x + product(*d0(h), *d0(w2))
    dgu = mx.matmul_swiglu_backward(*d0(dy), *d1(w2), (q, s), bits=block.bits)
    dn = product(*d0(dgu), *d1(w1))
    dx, dw, db = mx.layer_norm_backward(dn, (xq, xs), block.norm_w, mean, rstd)
    return y, [dy + dx, dw, db, product(*d1(dgu), *d1(n)), product(*d1(dy), *d1(h))]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("shape,dim,hidden", [((64,), 128, 192), ((2, 160), 256, 512),
                                              ((4, 256), 512, 1024), ((2048,), 256, 2112)])
def test_block(shape, dim, hidden, bits):
    block = block_of(dim, hidden, bits)
    x = rnd(*shape, dim, seed=1).requires_grad_()
    dy = rnd(*shape, dim, seed=2)
    y = block(x)
    y.backward(dy)
    got = [x.grad, block.norm_w.grad, block.norm_b.grad, block.w1.grad, block.w2.grad]
    flat, flat_dy = x.detach().reshape(-1, dim), dy.reshape(-1, dim)
    want, grads = by_hand(block, flat, flat_dy)
    assert torch.equal(y.detach().reshape(-1, dim), want)
    for a, b in zip(got, grads):
        assert torch.equal(a.reshape(b.shape), b)
    if bits == 8:
        want, grads = reference(flat, block.norm_w, block.norm_b, block.w1, block.w2, block.eps, flat_dy)

        def off(a, b):
            return float((a.detach().double().reshape(b.shape) - b).norm() / b.norm())
        assert off(y, want) < 4 * 2.0 ** -4
        for a, b, casts in zip(got, grads, (8, 8, 8, 7, 4)):
            assert off(a, b) < casts * 2.0 ** -4


def test_refusals():
    for bad in (dict(bits=4), dict(bits=16), dict(fused=True, bits=2)):
        with pytest.raises(ValueError, match="bits"):
            feed_forward.FeedForward(128, 128, **bad)
    with pytest.raises(ValueError, match="multiples of 64"):
        feed_forward.FeedForward(96, 128, fused=True, bits=4)
    block = feed_forward.FeedForward(64, 64, fused=True, bits=4)
    with pytest.raises(ValueError, match="tokens"):
        block(torch.zeros(32, 64, device="cuda", dtype=BF))
    x = rnd(64, 64).requires_grad_()
    g, = torch.autograd.grad(block(x).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.float().sum().backward()


def serve(x, gate, up, w2, bits):
    """A layer of a server on the rows of x, from weights cast once."""
    d0, product = (mx.cast_dim0, mx.matmul) if bits == 8 else (mx.cast_fp4_dim0, mx.matmul_fp4)
    h = mx.matmul_swiglu(*d0(x), *zip(gate, up), bits=bits)
    return product(*d0(h), *w2)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T,D,F", [(1, 512, 1408), (7, 256, 320), (300, 512, 2048)])
def test_serving_in_a_graph(T, D, F, bits):
    """Captured once, replayed on other tokens; rows do not depend on the others of the
    batch."""
    d0 = mx.cast_dim0 if bits == 8 else mx.cast_fp4_dim0
    gate, up, w2 = d0(rnd(F, D, seed=1)), d0(rnd(F, D, seed=2)), d0(rnd(D, F, seed=3))
    x = rnd(T, D, seed=4)
    want = serve(x, gate, up, w2, bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        serve(x, gate, up, w2, bits)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = serve(x, gate, up, w2, bits)
    graph.replay()
    assert torch.equal(y, want)
    x.copy_(rnd(T, D, seed=5))
    want = serve(x, gate, up, w2, bits)
    y.zero_()
    graph.replay()
    graph.replay()
    assert torch.equal(y, want)


@pytest.mark.parametrize("bits", [8, 4])
def test_a_step_in_a_graph(bits):
    """Forward and backward operators of a training step, captured and replayed."""
    T, D, F = 320, 256, 640
    block = block_of(D, F, bits)
    x, dy = rnd(T, D, seed=1), rnd(T, D, seed=2)
    want, grads = by_hand(block, x, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, got = by_hand(block, x, dy)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    for a, b in zip(got, grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [8, 4])
def test_autograds_step_in_a_graph(bits):
    """The block's own forward and backward pass captured, replayed on other tokens."""
    T, D, F = 320, 256, 640
    block, eager = block_of(D, F, bits), block_of(D, F, bits)
    x, dy = rnd(T, D, seed=1), rnd(T, D, seed=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            block.zero_grad(set_to_none=True)
            block(x).backward(dy)               # its graph is gone before the capture
    torch.cuda.current_stream().wait_stream(side)
    block.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x)
        y.backward(dy)
    for seed in (3, 5):
        x.copy_(rnd(T, D, seed=seed))
        dy.copy_(rnd(T, D, seed=seed + 1))
        graph.replay()
        eager.zero_grad(set_to_none=True)
        want = eager(x)
        want.backward(dy)
        assert torch.equal(y, want)
        for a, b in zip(block.parameters(), eager.parameters()):
            assert torch.equal(a.grad, b.grad)


def test_two_streams_at_once():
    """The same operators on two streams: nothing is shared between calls."""
    streams, want, got = [torch.cuda.Stream() for _ in range(2)], [], []
    blocks = [block_of(256, 1024, 8, seed=1), block_of(512, 640, 4, seed=2)]
    inputs = [(rnd(1024, 256, seed=3), rnd(1024, 256, seed=4)), (rnd(640, 512, seed=5), rnd(640, 512, seed=6))]
    for b, io in zip(blocks, inputs):
        want.append(by_hand(b, *io))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, b, io in zip(streams, blocks, inputs):
            with torch.cuda.stream(s):
                got.append(by_hand(b, *io))
    torch.cuda.synchronize()
    for i, (y, grads) in enumerate(got):
        assert torch.equal(y, want[i % 2][0])
        for a, b in zip(grads, want[i % 2][1]):
            assert torch.equal(a, b)
