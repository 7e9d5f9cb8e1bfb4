"""dw and db of the layer norm's backward pass where every term is a small whole
number: the sums are exact in fp32 whatever their order, so that one row left out
or counted twice shows.  mean 0 and rstd 1 make xh the input itself.
"""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
import plain64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()


def whole(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-7, 8, shape, generator=g, device="cuda").to(BF)


def check(x, dy, saved, wt):
    M, D = x.shape
    mean, rstd = torch.zeros(M, device="cuda"), torch.ones(M, device="cuda")
    _, dw, db = mx.layer_norm_backward(dy, saved, torch.ones(D, dtype=wt, device="cuda"), mean, rstd)
    assert 49 * M < 2 ** 24
    assert torch.equal(dw, (x.double() * dy.double()).sum(0).to(F32).to(wt))
    assert torch.equal(db, dy.double().sum(0).to(F32).to(wt))


@pytest.mark.parametrize("wt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D", [(1, 1), (7, 130), (10000, 640), (16640, 96), (6100, 1021), (1031, 1021),
                                 (2000, 4099), (330, 8190), (600, 4096), (4096, 4096), (2600, 5120),
                                 (153, 16384), (6100, 1504), (40001, 33)])
def test_from_bf16(M, D, wt):
    x, dy = whole((M, D), M + D), whole((M, D), M + D + 1)
    check(x, dy, x, wt)


# Whole numbers to 7 are e4m3 values at any scale that a block of them gets.
@pytest.mark.parametrize("wt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D", [(1, 32), (10000, 640), (16640, 96), (600, 4096), (2600, 5120), (153, 16384),
                                 (6100, 1504), (3100, 2304), (4096, 768)])
def test_from_the_saved_input(M, D, wt):
    x, dy = whole((M, D), M + D), whole((M, D), M + D + 1)
    q, s = mx.cast_dim0(x) if M % 32 == 0 else mx.layer_norm(x, torch.ones(D, device="cuda"), save=True)[3:]
    if M * D <= 4000000:
        assert torch.equal(plain64.mx_values(q, s), x.double())
    check(x, dy, (q, s), wt)
