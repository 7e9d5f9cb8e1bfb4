"""The 4-bit operators and the joined products through the bounds-checked build (as
test_gpu_training_bounds.py): no store refused, the release build's results; and their
abort paths."""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from test_gpu_training_bounds import checked, rnd, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def operand(R, K, bits, seed, size=1.0):
    x = (size * rnd((R, K), seed).float()).to(torch.bfloat16)
    return mx.cast_dim0(x) if bits == 8 else mx.cast_fp4_dim0(x)


@pytest.mark.parametrize("M,K", [(1, 32), (7, 160), (300, 96), (129, 5120), (2500, 1056)])
def test_rows(M, K):
    x = rnd((M, K), 1)
    same(lambda: mx.cast_fp4_dim0(x))
    a = mx.cast_fp4_dim0(x)
    same(lambda: mx.dequant_fp4(*a))


@pytest.mark.parametrize("M,K", [(32, 32), (160, 96), (2080, 1056)])
def test_tiles(M, K):
    x = rnd((M, K), 1)
    same(lambda: mx.cast_fp4_dim1(x))
    same(lambda: mx.cast_fp4_dim0_dim1(x))


@pytest.mark.parametrize("M,N,K", [(1, 1, 64), (130, 77, 192), (129, 136, 8256), (2056, 2320, 192),
                                   (2501, 1001, 192)])
def test_product(M, N, K):
    a, b = operand(M, K, 4, 1), operand(N, K, 4, 2)
    for dtype in (torch.bfloat16, torch.float32):
        same(lambda: mx.matmul_fp4(*a, *b, dtype))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,F,K", [(1, 32, 64), (130, 96, 192), (33, 1056, 4160), (1031, 2784, 192),
                                   (2304, 1184, 8256)])
def test_joined(M, F, K, bits):
    x, gate, up = operand(M, K, bits, 1), operand(F, K, bits, 2, 0.1), operand(F, K, bits, 3, 0.1)
    w = tuple(zip(gate, up))
    same(lambda: mx.matmul_swiglu(*x, *w, bits=bits))
    same(lambda: mx.matmul_swiglu(*x, *w, save=True, bits=bits))
    saved, gu = mx.matmul_swiglu(*x, *w, save=True, bits=bits)[1:], rnd((M, 2 * F), 4)
    for s in (saved, gu):
        same(lambda: mx.matmul_swiglu_backward(*x, *gate, s, bits=bits))


def gives_up(call, at):
    want = call()
    with checked():
        mx.mx_selftest_arm_stall(at)
        call()
        assert mx.mx_watchdog(clear=True) == 1
        got = call()
        assert mx.mx_watchdog(clear=True) == 0
        assert mx.mx_bounds_check(clear=True) == 0
    flat = lambda r: [r] if isinstance(r, torch.Tensor) else list(r)  # noqa: E731
    for a, b in zip(flat(got), flat(want)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("at", [0, 1, 3])
def test_casts_give_up(at):
    x = rnd((16640, 2560), 1)                # more than four tiles a CTA
    gives_up(lambda: mx.cast_fp4_dim0_dim1(x), at)
    gives_up(lambda: mx.cast_fp4_dim1(x), at)
    gives_up(lambda: mx.cast_fp4_dim0(x), at)
    a = mx.cast_fp4_dim0(x)
    gives_up(lambda: mx.dequant_fp4(*a), at)


def calls(M, F, K, bits):
    x, gate, up = operand(M, K, bits, 1), operand(F, K, bits, 2, 0.02), operand(F, K, bits, 3, 0.02)
    gu = rnd((M, 2 * F), 4)
    saved = mx.cast_dim0(gu)
    yield lambda: mx.matmul_swiglu(*x, *zip(gate, up), bits=bits)
    yield lambda: mx.matmul_swiglu(*x, *zip(gate, up), save=True, bits=bits)
    yield lambda: mx.matmul_swiglu_backward(*x, *gate, gu, bits=bits)
    yield lambda: mx.matmul_swiglu_backward(*x, *gate, saved, bits=bits)
    if bits == 4:
        yield lambda: mx.matmul_fp4(*x, *gate)
        yield lambda: mx.matmul_fp4(*x, *gate, torch.float32)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("at", [0, 1, 5])
def test_products_in_tiles_give_up(at, bits):
    """A load that never comes, with a whole contraction and with one cut among eight CTAs, of
    eight loads a CTA at least."""
    for shape in ((600, 1152, 2048), (64, 64, 16384)):
        for call in calls(*shape, bits):
            gives_up(call, at)


@pytest.mark.parametrize("at,bits", [(0, 4), (5, 8), (9, 4)])
def test_products_in_pairs_give_up(at, bits):
    for call in calls(2304, 2304, 2048, bits):
        gives_up(call, at)
