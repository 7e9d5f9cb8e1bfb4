"""The product of MX-FP4 operands on the GPU against the same sum in 64 bits.  Tolerance:
plain_fp4.product, plus half a unit in the last place for a bf16 result."""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from plain64 import blocked_at
from plain_fp4 import BF16, product

pytestmark = pytest.mark.gpu

GUARD = 256
TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()
    assert mx.mx_watchdog(clear=True) == 0
    yield
    torch.cuda.synchronize()
    assert mx.mx_watchdog(clear=True) == 0


def operand(R, K, seed, lo=110, hi=144):
    """Random codes and scales; the scale buffer's padding holds 0xFF, which no result may
    depend on."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 256, (R, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.full((mx.mx_blocked_bytes(R, K // 32),), 255, dtype=torch.uint8, device="cuda")
    at = blocked_at(R, K // 32, "cuda")
    s[at] = torch.randint(lo, hi, at.shape, generator=g, device="cuda").to(torch.uint8)
    return q, s


def run(a, b, dtype):
    M, N = a[0].shape[0], b[0].shape[0]
    buf = torch.full((M * N + GUARD,), 5.0, dtype=dtype, device="cuda")
    out = buf[:M * N].view(M, N)
    mx.mx_matmul_fp4(*a, *b, out)
    torch.cuda.synchronize()
    assert bool((buf[M * N:] == 5.0).all()), "written past the end"
    return out


def check(a, b, got):
    want, _, tol = product(a, b, 4)
    if got.dtype == torch.bfloat16:
        tol = tol * (1 + BF16) + BF16 * want.abs()
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), "%d of %d values off" % (int(bad.sum()), bad.numel())


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [
    (128, 128, 256), (1, 1, 64), (1, 128, 64), (128, 1, 64), (127, 129, 128), (129, 127, 192), (31, 33, 2112),
    (160, 96, 1024), (1, 1000, 4160), (300, 1000, 576), (257, 255, 1088), (256, 256, 256),
    (512, 512, 512), (1000, 1032, 320), (7, 4096, 512), (2050, 1030, 640)])
def test_matches_64_bits(M, N, K, dtype):
    a, b = operand(M, K, M + 7 * N + K), operand(N, K, M + 3 * N + K + 1)
    check(a, b, run(a, b, dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(32, 32, 16640), (4096, 2304, 192), (3000, 5000, 4224),
                                   (2304, 4352, 8256)])
def test_long_and_wide(M, N, K, dtype):
    a, b = operand(M, K, K), operand(N, K, K + 1)
    check(a, b, run(a, b, dtype))


@pytest.mark.parametrize("M,N,K", [(64, 64, 65536), (384, 256, 16384), (2304, 4352, 16640)])
def test_long_fp32_sums_of_equal_signs(M, N, K):
    """Sums that only grow: cut-off bits do not cancel, and fp32's own error is kept by
    adding runs of 4096 steps in fp32 (4e-7 a run at one sign, a rounding a run)."""
    a, b = operand(M, K, 1, 120, 136), operand(N, K, 2, 120, 136)
    a, b = (a[0] & 0x77, a[1]), (b[0] & 0x77, b[1])
    got = run(a, b, torch.float32)
    want, size, _ = product(a, b, 4)
    off = (got.double() - want).norm() / want.norm()
    # 64 instructions a run cut at most 2^-23 each of a sum that grows evenly, half of it on
    # average, the runs' additions 2^-24 of theirs.
    assert float(off) < 32 * 2.0 ** -23 + K / 4096 * 2.0 ** -25


@pytest.mark.parametrize("M,N,K", [(3, 200, 1024), (300, 520, 448), (2304, 2304, 512)])
def test_nan_scales_reach_their_rows_only(M, N, K):
    a, b = operand(M, K, 5), operand(N, K, 6)
    s = a[1].clone()
    s[blocked_at(M, K // 32, "cuda")[M // 2, K // 64]] = 255
    want = run(a, b, torch.float32)
    got = run((a[0], s), b, torch.float32)
    assert bool(torch.isnan(got[M // 2]).all())
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(got[keep], want[keep])


def test_one_hot_operands():
    """Every element, scale and place of the contraction, one at a time: exact."""
    K = 512
    a_codes = torch.zeros(K, K, dtype=torch.uint8, device="cuda")
    i = torch.arange(K, device="cuda")
    a_codes[i, i] = (1 + i % 15).to(torch.uint8)
    q = a_codes[:, 0::2] | (a_codes[:, 1::2] << 4)
    s = torch.full((mx.mx_blocked_bytes(K, K // 32),), 255, dtype=torch.uint8, device="cuda")
    at = blocked_at(K, K // 32, "cuda")
    s[at] = (100 + (7 * i[:, None] + at % 13) % 50).to(torch.uint8)
    b = operand(640, K, 3)
    got = run((q, s), b, torch.float32)
    assert torch.equal(got.double(), product((q, s), b, 4)[0])


def test_against_the_cast_of_equal_values():
    """The same numbers as MX-FP8 give the same exact sums."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randint(-3, 4, (200, 320), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(-3, 4, (136, 320), generator=g, device="cuda").to(torch.bfloat16)
    x[:, ::32], w[:, ::32] = 4, 4
    got = mx.matmul_fp4(*mx.cast_fp4_dim0(x), *mx.cast_fp4_dim0(w), torch.float32)
    assert torch.equal(got, mx.matmul(*mx.cast_dim0(x), *mx.cast_dim0(w), torch.float32))
    assert torch.equal(got.double(), x.double() @ w.double().t())


def test_the_three_products_of_a_linear_layer():
    T, K, N = 192, 256, 320
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w, dy = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
                for s in ((T, K), (N, K), (T, N)))
    x0, xs0, x1, xs1 = mx.cast_fp4_dim0_dim1(x)
    w0, ws0, w1, ws1 = mx.cast_fp4_dim0_dim1(w)
    d0, ds0, d1, ds1 = mx.cast_fp4_dim0_dim1(dy)
    for a, b in (((x0, xs0), (w0, ws0)), ((d0, ds0), (w1, ws1)), ((d1, ds1), (x1, xs1))):
        for dtype in TYPES:
            check(a, b, mx.matmul_fp4(*a, *b, dtype))


def test_repeats_itself():
    a, b = operand(700, 2112, 1), operand(900, 2112, 2)
    want = run(a, b, torch.float32)
    for _ in range(3):
        assert torch.equal(run(a, b, torch.float32), want)


@pytest.mark.parametrize("N", [40960, 40963])
def test_offsets_past_32_bits(N):
    """Results past 2^31 values and 2^33 bytes, through tensor maps and rows, on sampled rows."""
    M, K = 65536, 64
    a, b = operand(M, K, 1), operand(N, K, 2)
    got = mx.matmul_fp4(*a, *b, torch.float32)
    rows = torch.tensor([0, 1, 32767, 52427, 52428, 52429, 65535], device="cuda")
    part = a[0][rows].contiguous(), mx.scales_to_blocked(a[1][blocked_at(M, K // 32, "cuda")[rows]])
    want, _, tol = product(part, b, 4)
    assert bool(((got[rows].double() - want).abs() <= tol).all())
