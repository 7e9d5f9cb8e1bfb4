"""The feed-forward block on the GPU: its output and gradients against 64 bits of
the unquantised block.

Tolerance: an MX cast moves a value by at most 2^-4 of it (half a unit in the last
of e4m3's four bits; values that saturate, above 448 / 256 of the block's power of
two, by at most 2^-3).  n casts on the way to a result leave it within n 2^-4 of
its 2-norm, the directions of the errors being as good as independent.
"""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from mxfp8_block_scaled_dim0_gb300 import feed_forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()
    yield
    torch.cuda.synchronize()
    assert mx.mx_watchdog(clear=True) == 0


def reference(x, norm_w, norm_b, w1, w2, eps, dy):
    args = [t.detach().double().requires_grad_() for t in (x, norm_w, norm_b, w1, w2)]
    x, nw, nb, a, b = args
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps) ** -0.5
    g, u = (((x - mean) * rstd * nw + nb) @ a.t()).chunk(2, -1)
    y = x + (g * torch.sigmoid(g) * u) @ b.t()
    y.backward(dy.double())
    return y.detach(), [t.grad for t in args]


@pytest.mark.parametrize("shape,dim,hidden", [((64,), 96, 160), ((2, 160), 256, 512),
                                              ((4, 256), 512, 1024)])
def test_block(shape, dim, hidden):
    torch.manual_seed(3)
    block = feed_forward.FeedForward(dim, hidden)
    with torch.no_grad():
        block.norm_w.add_(0.2 * torch.randn_like(block.norm_w))
        block.norm_b.add_(0.2 * torch.randn_like(block.norm_b))
    x = torch.randn(*shape, dim, device="cuda").to(torch.bfloat16).requires_grad_()
    dy = torch.randn(*shape, dim, device="cuda").to(torch.bfloat16)
    y = block(x)
    y.backward(dy)
    got = [x.grad, block.norm_w.grad, block.norm_b.grad, block.w1.grad, block.w2.grad]
    flat = x.detach().reshape(-1, dim)
    want, grads = reference(flat, block.norm_w, block.norm_b, block.w1, block.w2, block.eps,
                            dy.reshape(-1, dim))

    def off(a, b):
        return float((a.detach().double().reshape(b.shape) - b).norm() / b.norm())

    # casts on the way: n, w1, h, w2 to y; dy, w2, gu, dgu, w1, x to dx, dw and db
    # (through the saved gu, n and w1 again); dy, h (n, w1) to dw2; these and gu to dw1
    assert off(y, want) < 4 * 2.0 ** -4
    for g, w, casts in zip(got, grads, (8, 8, 8, 7, 4)):
        assert g.dtype == (torch.float32 if g.dim() == 1 else torch.bfloat16)
        assert off(g, w) < casts * 2.0 ** -4


def test_keeps_half_the_bytes():
    T, D, F = 640, 256, 512
    block = feed_forward.FeedForward(D, F)
    x = torch.randn(T, D, device="cuda").to(torch.bfloat16)
    y = feed_forward._Block.apply(x, block.norm_w, block.norm_b, block.w1, block.w2, block.eps)
    of_weights = {(D, 2 * F), (F, D)}
    kept = sum(t.nbytes for t in y.grad_fn.saved_tensors
               if t.dtype == torch.uint8 and tuple(t.shape) not in of_weights)
    kept -= mx.mx_blocked_bytes(D, 2 * F // 32) + mx.mx_blocked_bytes(F, D // 32)
    assert kept == T * (2 * D + 3 * F) * 33 // 32


def test_trains():
    torch.manual_seed(1)
    block = feed_forward.FeedForward(128, 256)
    x = torch.randn(256, 128, device="cuda").to(torch.bfloat16)
    target = torch.randn(256, 128, device="cuda").to(torch.bfloat16)
    opt = torch.optim.SGD(block.parameters(), lr=1.0)
    losses = []
    for _ in range(20):
        loss = (block(x).float() - target.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    assert losses[-1] < 0.9 * losses[0]


def test_refusals():
    with pytest.raises(ValueError, match="multiples of 32"):
        feed_forward.FeedForward(100, 64)
    block = feed_forward.FeedForward(64, 64)
    with pytest.raises(ValueError, match="tokens"):
        block(torch.zeros(5, 64, device="cuda", dtype=torch.bfloat16))


def test_calls_from_a_new_thread():
    """A thread that has made no CUDA call yet (autograd runs backward passes on
    such ones): the first call there needs tensor maps, a driver call."""
    import threading
    x = torch.randn(160, 96, device="cuda").to(torch.bfloat16)
    want, got, failed = mx.cast_dim0_dim1(x), [], []

    def work():
        try:
            got.append(mx.cast_dim0_dim1(x))
        except Exception as e:
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not failed, failed
    torch.cuda.synchronize()
    for a, b in zip(got[0], want):
        assert torch.equal(a, b)
