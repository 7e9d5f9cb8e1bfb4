"""Seeded random shapes through the 4-bit operators and the joined products, against 64
bits: sizes and tolerances as in their own tests."""
import random

import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
import test_gpu_fp4_casts as casts
import test_gpu_matmul_fp4 as products
import test_gpu_matmul_swiglu as joined

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()
    yield
    torch.cuda.synchronize()
    assert mx.mx_watchdog(clear=True) == 0


def size(rng, most, step=1):
    """Sizes spread over their logarithm, multiples of step."""
    return max(step, int(most ** rng.random()) // step * step)


@pytest.mark.parametrize("seed", range(24))
def test_casts(seed):
    rng = random.Random(seed)
    M, K = size(rng, 3000), size(rng, 2000, 32)
    casts.check(casts.rnd(M, K, seed), "0")
    M = max(32, M // 32 * 32)
    casts.check(casts.rnd(M, K, seed), rng.choice(["1", "01"]))
    casts.test_dequant(size(rng, 3000), size(rng, 2000, 32))


@pytest.mark.parametrize("seed", range(32))
def test_products(seed):
    rng = random.Random(100 + seed)
    M, N, K = size(rng, 4000), size(rng, 3000), size(rng, 4000, 64)
    a, b = products.operand(M, K, seed), products.operand(N, K, seed + 1)
    products.check(a, b, products.run(a, b, rng.choice(products.TYPES)))


@pytest.mark.parametrize("seed", range(40))
def test_joined(seed):
    rng = random.Random(200 + seed)
    bits = rng.choice([8, 4])
    M, F, K = size(rng, 4000), size(rng, 3000, 32), size(rng, 6000, 32 if bits == 8 else 64)
    joined.forward(M, F, K, bits, rng.random() < 0.6, seed)
    M, F, K = size(rng, 4000), size(rng, 3000, 32), size(rng, 4000, 32 if bits == 8 else 64)
    joined.backward(M, F, K, bits, rng.choice([8, 16]), seed)
