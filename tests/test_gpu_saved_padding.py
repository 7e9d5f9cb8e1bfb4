"""Scale bytes that belong to no block reach no result: the buffers' padding (rows
past the matrix, scales past a row) filled with 0xFF, which as a scale is NaN."""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
import plain64

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()


def rnd(shape, seed, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def spoiled(s, R, C):
    """Blocked scales of an R x C/32 matrix with every byte of padding 0xFF."""
    at = plain64.blocked_at(R, C // 32, "cuda")
    t = torch.full_like(s, 255)
    t[at] = s[at]
    assert not torch.equal(t, s)
    return t


# Widths of one to three blocks past a multiple of four, 8 to 32 values a thread, one
# group and many; rows that end a scale tile and rows that do not.
@pytest.mark.parametrize("M,D", [(128, 32), (5, 64), (130, 96), (128, 160), (300, 416), (40, 1056),
                                 (3, 4128), (1300, 8224), (6100, 1504), (2500, 2272), (2, 16352)])
def test_layer_norm_backward(M, D):
    x, dy, w = rnd((M, D), 1), rnd((M, D), 2), rnd((D,), 3, torch.float32)
    _, mean, rstd, q, s = mx.layer_norm(x, w, save=True)
    want = mx.layer_norm_backward(dy, (q, s), w, mean, rstd)
    got = mx.layer_norm_backward(dy, (q, spoiled(s, M, D)), w, mean, rstd)
    for a, b in zip(got, want):
        assert bool(torch.isfinite(b).all()) and torch.equal(a, b)


@pytest.mark.parametrize("M,F", [(128, 32), (130, 96), (7, 224), (300, 1056)])
def test_swiglu_backward(M, F):
    gu, dh = rnd((M, 2 * F), 1), rnd((M, F), 2)
    _, q, s = mx.swiglu(gu, save=True)
    want = mx.swiglu_backward(dh, (q, s))
    got = mx.swiglu_backward(dh, (q, spoiled(s, M, 2 * F)))
    assert bool(torch.isfinite(want).all()) and torch.equal(got, want)


def test_nan_scales_of_blocks_still_count():
    M, D = 70, 96
    x, dy, w = rnd((M, D), 1), rnd((M, D), 2), rnd((D,), 3, torch.float32)
    _, mean, rstd, q, s = mx.layer_norm(x, w, save=True)
    s[plain64.blocked_at(M, 3, "cuda")[5, 2]] = 255
    dx, dw, db = mx.layer_norm_backward(dy, (q, s), w, mean, rstd)
    nan = torch.isnan(dx)
    assert bool(nan[5].all()) and int(nan.sum()) == D
    assert bool(torch.isnan(dw[64:]).all()) and bool(torch.isfinite(dw[:64]).all())
    assert bool(torch.isfinite(db).all())
