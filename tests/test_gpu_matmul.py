"""The product of MX operands on the GPU against the same sum in 64 bits.

Tolerance, fixed by the arithmetic: every product of two e4m3 values times two
powers of two is exact, the tensor core adds 32 of them and the running sum at
a time, and each such addition loses at most one unit of the last of 24 bits
of the largest magnitude that takes part, which sum |a b| bounds; with the up
to 32 terms of one addition cut off separately,

    |c - c64| <= (K / 32 + 32) 2^-23 sum_k |a_k b_k|,

plus half a unit in the last place for a bf16 result.
"""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from plain64 import blocked_at, mx_values

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
    """Random finite e4m3 bytes and scales; the scale buffer's padding holds
    0xFF, which no result may depend on."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 256, (R, K), generator=g, device="cuda", dtype=torch.uint8)
    q[(q & 127) == 127] = 0x31
    s = torch.full((mx.mx_blocked_bytes(R, K // 32),), 255, dtype=torch.uint8, device="cuda")
    at = blocked_at(R, K // 32, "cuda")
    s[at] = torch.randint(lo, hi, at.shape, generator=g, device="cuda").to(torch.uint8)
    return q, s


def product(a, b, dtype):
    """mx_matmul into a guarded buffer."""
    M, N = a[0].shape[0], b[0].shape[0]
    buf = torch.full((M * N + GUARD,), 5.0, dtype=dtype, device="cuda")
    out = buf[:M * N].view(M, N)
    mx.mx_matmul(*a, *b, out)
    torch.cuda.synchronize()
    assert bool((buf[M * N:] == 5.0).all()), "written past the end"
    return out


def check(a, b, got):
    K = a[0].shape[1]
    va, vb = mx_values(*a), mx_values(*b)
    want = va @ vb.t()
    tol = (K / 32 + 32) * 2.0 ** -23 * (va.abs() @ vb.abs().t())
    if got.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    bad = (got.double() - want).abs() > tol
    assert not bool(bad.any()), "%d of %d values off" % (int(bad.sum()), bad.numel())


SHAPES = [
    (1, 1, 32), (1, 128, 32), (128, 1, 64), (127, 129, 96), (128, 128, 128), (129, 127, 160),
    (31, 33, 2080), (160, 96, 1024), (1, 1000, 4128), (300, 1000, 544), (257, 255, 1056),
    (256, 256, 256), (512, 512, 512), (1000, 1032, 288), (7, 4096, 512), (2050, 1030, 640),
]


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matches_64_bits(M, N, K, dtype):
    a, b = operand(M, K, M + 7 * N + K), operand(N, K, M + 3 * N + K + 1)
    check(a, b, product(a, b, dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(32, 32, 16640), (4096, 2304, 160), (3000, 5000, 4192),
                                   (2304, 4352, 8224)])
def test_long_and_wide(M, N, K, dtype):
    a, b = operand(M, K, K), operand(N, K, K + 1)
    check(a, b, product(a, b, dtype))


@pytest.mark.parametrize("by_column", ["a", "b", "ab"])
@pytest.mark.parametrize("M,N,K", [(16, 16, 32), (144, 272, 96), (128, 1040, 544), (2064, 2320, 352),
                                   (16, 5120, 2080)])
def test_operands_stored_by_column(M, N, K, by_column):
    a, b = operand(M, K, M + N + K), operand(N, K, M + N + K + 1)
    want = product(a, b, torch.float32)
    if "a" in by_column:
        a = (a[0].t().contiguous().t(), a[1])
    if "b" in by_column:
        b = (b[0].t().contiguous().t(), b[1])
    got = product(a, b, torch.float32)
    check(a, b, got)
    assert torch.equal(got, want)


def test_long_sum_of_equal_terms():
    """A sum that only grows, over 16384 steps: cut-off bits do not cancel."""
    M, N, K = 384, 256, 16384
    a, b = operand(M, K, 1), operand(N, K, 2)
    a[0].fill_(0x39)                 # 1.125
    b[0].fill_(0x3B)                 # 1.375
    for s in (a[1], b[1]):
        s.fill_(127)
    check(a, b, product(a, b, torch.float32))


@pytest.mark.parametrize("M,N,K", [(130, 140, 96), (700, 900, 2080)])
def test_same_bits_every_time(M, N, K):
    a, b = operand(M, K, 5), operand(N, K, 6)
    first = product(a, b, torch.float32).view(torch.int32).clone()
    for _ in range(3):
        assert torch.equal(product(a, b, torch.float32).view(torch.int32), first)


@pytest.mark.parametrize("M,N,K", [(140, 150, 160), (600, 520, 1056)])
def test_nan_stays_in_its_row_and_column(M, N, K):
    a, b = operand(M, K, 8), operand(N, K, 9)
    a[0][3, 40] = 0x7F                                                # NaN element
    a[1][blocked_at(M, K // 32, "cuda")[M - 1, K // 32 - 1]] = 255    # NaN scale
    b[0][N - 1, K - 1] = 0xFF
    got = product(a, b, torch.float32)
    nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    nan[3], nan[M - 1], nan[:, N - 1] = True, True, True
    assert torch.equal(torch.isnan(got), nan)
    rest = (mx_values(*a) @ mx_values(*b).t())[~nan]
    assert bool(((got[~nan].double() - rest).abs() <= 1e-4 * rest.abs().max()).all())


def test_range_ends():
    """The largest scales overflow to infinity with the sum's sign; the smallest
    ones with the largest give ordinary numbers."""
    K = 64
    a, b = operand(40, K, 1), operand(50, K, 2)
    a[0].fill_(0x7E)
    b[0].fill_(0x7E)                     # 448
    b[0][25:] = 0xFE
    sa, sb = a[1], b[1]
    sa.fill_(254)
    sb.fill_(254)
    got = product(a, b, torch.bfloat16).float()
    assert bool((got[:, :25] == float("inf")).all()) and bool((got[:, 25:] == -float("inf")).all())
    sb.fill_(0)                          # 2^-127 times 2^127
    got = product(a, b, torch.float32)
    want = 448.0 * 448.0 * K
    assert bool((got[:, :25] == want).all()) and bool((got[:, 25:] == -want).all())


def test_outputs_beyond_32_bit_offsets():
    """M N above 2^31: the last rows land at their own addresses."""
    M, N, K = 70016, 32768, 32
    a, b = operand(M, K, 3), operand(N, K, 4)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    mx.mx_matmul(*a, *b, out)
    va, vb = mx_values(*a), mx_values(*b)
    for r in (0, 35000, 65535, 65536, M - 1):
        want = vb @ va[r]
        assert bool(((out[r].double() - want).abs() <= 2.0 ** -8 * want.abs()
                     + 33 * 2.0 ** -23 * (vb.abs() @ va[r].abs())).all()), r
    del out


def test_gradient_products_of_a_linear_layer():
    """dx and dW of y = x W^T from the casts, against the same products of what
    the casts stand for."""
    T, N, K = 416, 352, 288
    g = torch.Generator(device="cuda").manual_seed(11)
    x, w, dy = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
                for s in ((T, K), (N, K), (T, N)))
    x0, x1 = mx.cast_dim0(x), mx.cast_dim1(x)
    w0, w1 = mx.cast_dim0(w), mx.cast_dim1(w)
    d0, d1 = mx.cast_dim0(dy), mx.cast_dim1(dy)
    for a, b in ((x0, w0), (d0, w1), (d1, x1)):
        got = mx.matmul(*a, *b)
        assert got.dtype == torch.bfloat16
        check(a, b, got)
    full = (dy.double().t() @ x.double())
    got = mx.matmul(*d1, *x1, torch.float32).double()
    # each operand is within 2^-4 of its value in the 2-norm over a block
    assert float((got - full).norm() / full.norm()) < 2 * 2.0 ** -4


def test_on_another_stream():
    a, b = operand(300, 512, 1), operand(200, 512, 2)
    want = mx.matmul(*a, *b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = mx.matmul(*a, *b, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = mx.matmul(*a, *b)
    s.synchronize()
    assert torch.equal(got, want)


def test_in_a_cuda_graph():
    a, b = operand(260, 512, 1), operand(270, 512, 2)
    out = torch.zeros((260, 270), dtype=torch.float32, device="cuda")
    mx.mx_matmul(*a, *b, out)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.mx_matmul(*a, *b, out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_refusals():
    a, b = operand(64, 64, 1), operand(96, 64, 2)
    out = torch.zeros((64, 96), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="equal rows"):
        mx.mx_matmul(*a, *operand(96, 128, 2), out)
    with pytest.raises(ValueError, match="shape"):
        mx.mx_matmul(*a, *b, out[:32])
    with pytest.raises(TypeError, match="out"):
        mx.mx_matmul(*a, *b, out.half())
    with pytest.raises(ValueError, match="contiguous"):
        mx.mx_matmul(torch.zeros((64, 128), dtype=torch.uint8, device="cuda")[:, :64], a[1], *b, out)
    with pytest.raises(ValueError, match="sb_blk holds"):
        mx.mx_matmul(*a, b[0], b[1][:100], out)
    with pytest.raises(ValueError, match="CUDA"):
        mx.mx_matmul(*a, *b, out.cpu())
    q = torch.zeros((64, 48), dtype=torch.uint8, device="cuda")
    with pytest.raises(mx.MXError) as e:
        mx.mx_matmul(q, a[1], torch.zeros((96, 48), dtype=torch.uint8, device="cuda"), b[1], out)
    assert e.value.code == mx.MX_ERR_SHAPE


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [1001, 1002, 1004, 1023, 1026])
@pytest.mark.parametrize("M,K", [(2501, 160), (2470, 4192)])
def test_rows_off_the_boundary(M, N, K, dtype):
    """Enough tiles for the pairs, rows of results that begin anywhere."""
    a, b = operand(M, K, M + N), operand(N, K, N + 1)
    check(a, b, product(a, b, dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(500, 701, 800), (161, 1022, 1024), (16640, 333, 64), (33, 2817, 96)])
def test_few_tiles_off_the_boundary(M, N, K, dtype):
    a, b = operand(M, K, M + N), operand(N, K, N + 1)
    check(a, b, product(a, b, dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(160, 1024, 1024), (160, 1000, 4096), (79, 4624, 1856), (126, 600, 1600),
                                   (499, 40, 1984), (25, 1736, 864), (38, 2312, 2112), (512, 512, 512),
                                   (1, 200, 224), (130, 72, 8224)])
def test_few_tiles(M, N, K, dtype):
    """Tiles of 64 columns and of 128, whole and cut."""
    a, b = operand(M, K, M + N), operand(N, K, N + 1)
    check(a, b, product(a, b, dtype))
