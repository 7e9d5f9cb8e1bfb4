"""fp32 products over long contractions, from every kernel that the sizes choose.

The tensor core's accumulator cuts bits off at each addition of 32 steps, an error
that grows with the length of a sum, so sums for an fp32 result run over 4096
steps at most and are added up in fp32.  The documented error of such a run is
3.7e-7 in the 2-norm, for operands of random signs; 5e-7 leaves a third.  For
operands of one sign no error cancels: each of a run's 128 additions, and each of
the 32 terms of one, loses at most one unit of the last of 24 bits of the run's
sum, and R runs are added with 2^-24 each: (160 + R) 2^-23 of the sum.
"""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from plain64 import blocked_at, mx_values
from test_gpu_training_bounds import checked

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()
    assert mx.mx_watchdog(clear=True) == 0
    yield
    torch.cuda.synchronize()
    assert mx.mx_watchdog(clear=True) == 0


def operand(R, K, seed, one_sign=False):
    """Normal deviates cast along their rows, or random bytes of one sign."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    if not one_sign:
        return mx.cast_dim0(torch.randn((R, K), generator=g, device="cuda").to(torch.bfloat16))
    q = torch.randint(0x20, 0x78, (R, K), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.full((mx.mx_blocked_bytes(R, K // 32),), 255, dtype=torch.uint8, device="cuda")
    s[blocked_at(R, K // 32, "cuda")] = 127
    return q, s


# One CTA a tile, of 128 columns and of 64; two to eight CTAs a tile; CTA pairs.
SHAPES = [(1536, 1536, 16640), (1024, 1000, 16640), (100, 70, 8224), (32, 32, 131072),
          (256, 256, 131072), (1, 1000, 65536), (520, 610, 32800), (2304, 4352, 16640)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_random_signs(M, N, K):
    a, b = operand(M, K, 1), operand(N, K, 2)
    want = mx_values(*a) @ mx_values(*b).t()
    got = mx.matmul(*a, *b, torch.float32).double()
    assert float((got - want).norm() / want.norm()) < 5e-7


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_one_sign(M, N, K):
    a, b = operand(M, K, 3, True), operand(N, K, 4, True)
    want = mx_values(*a) @ mx_values(*b).t()
    got = mx.matmul(*a, *b, torch.float32).double()
    runs = (K + 4095) // 4096 + 8
    assert float(((got - want).abs() / want).max()) <= (160 + runs) * 2.0 ** -23


@pytest.mark.parametrize("M,N,K", [(144, 160, 16640), (1040, 528, 12320)])
def test_the_storage_order_changes_no_bit(M, N, K):
    a, b = operand(M, K, 5), operand(N, K, 6)
    want = mx.matmul(*a, *b, torch.float32)
    at, bt = (a[0].t().contiguous().t(), a[1]), (b[0].t().contiguous().t(), b[1])
    for x, y in ((at, b), (a, bt), (at, bt)):
        assert torch.equal(mx.matmul(*x, *y, torch.float32), want)
    for _ in range(3):
        assert torch.equal(mx.matmul(*a, *b, torch.float32), want)


@pytest.mark.parametrize("M,N,K", [(300, 701, 8320), (1500, 1022, 16640)])
def test_rows_off_the_boundary(M, N, K):
    a, b = operand(M, K, 7), operand(N, K, 8)
    buf = torch.full((M * N + 256,), 5.0, device="cuda")
    mx.mx_matmul(*a, *b, buf[:M * N].view(M, N))
    assert bool((buf[M * N:] == 5.0).all()), "written past the end"
    want = mx_values(*a) @ mx_values(*b).t()
    assert float((buf[:M * N].view(M, N).double() - want).norm() / want.norm()) < 5e-7


@pytest.mark.parametrize("M,N,K", [(1100, 1100, 8320), (64, 128, 65536)])
def test_checked_build(M, N, K):
    """Sums of several runs: no store out of bounds; a load that never comes, in the
    first run, at its end and in a later one, ends the call."""
    a, b = operand(M, K, 9), operand(N, K, 10)
    want = mx.matmul(*a, *b, torch.float32)
    with checked():
        assert torch.equal(mx.matmul(*a, *b, torch.float32), want)
        for at in (0, 31, 33, 60):
            mx.mx_selftest_arm_stall(at)
            mx.matmul(*a, *b, torch.float32)
            assert mx.mx_watchdog(clear=True) == 1
            assert torch.equal(mx.matmul(*a, *b, torch.float32), want)
            assert mx.mx_watchdog(clear=True) == 0
        assert mx.mx_bounds_check(clear=True) == 0
