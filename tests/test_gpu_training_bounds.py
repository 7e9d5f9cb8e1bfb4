"""The training operators through the bounds-checked build: every store of their
threads is checked against its buffer, none may be refused, and the results are
those of the release build.  The stall hook drives the abort paths of the kernels
that wait: the call returns, the watchdog word is set, the next call works."""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from mxfp8_block_scaled_dim0_gb300 import build as mxbuild

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class checked:
    """The bounds-checked library in place of the release one."""

    def __enter__(self):
        self.saved = (mx.LIB_PATH, mx._LIB)
        mx.LIB_PATH, mx._LIB = mxbuild.build(bounds=True), None
        mx.mx_bounds_check(clear=True)
        mx.mx_watchdog(clear=True)

    def __exit__(self, *exc):
        torch.cuda.synchronize()
        mx.LIB_PATH, mx._LIB = self.saved


def rnd(shape, seed, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def same(call):
    want = call()
    with checked():
        got = call()
        torch.cuda.synchronize()
        assert mx.mx_bounds_check(clear=True) == 0
        assert mx.mx_watchdog(clear=True) == 0
    flat = lambda r: [r] if isinstance(r, torch.Tensor) else list(r)  # noqa: E731
    for a, b in zip(flat(got), flat(want)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("M,D", [(1, 1), (7, 1021), (300, 250), (33, 4100), (2, 16383), (130, 96),
                                 (40, 5120), (3, 16384), (700, 512)])
def test_layer_norm(M, D):
    x, dy, w, b = rnd((M, D), 1), rnd((M, D), 2), rnd((D,), 3, torch.float32), rnd((D,), 4, torch.float32)
    same(lambda: mx.layer_norm(x, w, b))
    _, mean, rstd = mx.layer_norm(x, w, b)
    same(lambda: mx.layer_norm_backward(dy, x, w, mean, rstd))
    same(lambda: mx.layer_norm_backward(dy, x, w.to(BF), mean, rstd))
    if D % 32 == 0:
        same(lambda: mx.layer_norm(x, w, b, save=True))
        saved = mx.layer_norm(x, w, b, save=True)[3:]
        same(lambda: mx.layer_norm_backward(dy, saved, w, mean, rstd))


@pytest.mark.parametrize("M,F", [(1, 1), (5, 33), (9, 62), (130, 32), (129, 96), (64, 128), (3, 4096),
                                 (12501, 4096)])
def test_swiglu(M, F):
    gu, dh = rnd((M, 2 * F), 1), rnd((M, F), 2)
    same(lambda: mx.swiglu(gu))
    same(lambda: mx.swiglu_backward(dh, gu))
    if F % 32 == 0:
        same(lambda: mx.swiglu(gu, save=True))
        saved = mx.swiglu(gu, save=True)[1:]
        same(lambda: mx.swiglu_backward(dh, saved))


@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (130, 77, 96), (129, 136, 4128), (2056, 2320, 160)])
def test_matmul(M, N, K):
    a, b = mx.cast_dim0(rnd((M, K), 1)), mx.cast_dim0(rnd((N, K), 2))
    for dtype in (BF, torch.float32):
        same(lambda: mx.matmul(*a, *b, dtype))


@pytest.mark.parametrize("at", [0, 1, 5])
def test_matmul_gives_up(at):
    """A load that never comes, in the one-tile kernel (with and without a cut
    contraction) and in the pair kernel."""
    for M, N, K in ((128, 128, 1024), (64, 128, 16384), (2304, 4096, 1024)):
        a, b = mx.cast_dim0(rnd((M, K), 1)), mx.cast_dim0(rnd((N, K), 2))
        want = mx.matmul(*a, *b)
        with checked():
            mx.mx_selftest_arm_stall(at)
            mx.matmul(*a, *b)
            assert mx.mx_watchdog(clear=True) == 1
            assert torch.equal(mx.matmul(*a, *b), want)
            assert mx.mx_watchdog(clear=True) == 0
            assert mx.mx_bounds_check(clear=True) == 0


@pytest.mark.parametrize("at", [0, 1, 4])
@pytest.mark.parametrize("D", [96, 1021, 4096])
def test_layer_norm_gives_up(D, at):
    M = 6000 if D > 2000 else 40000          # five rows a group at least
    x, dy, w = rnd((M, D), 1), rnd((M, D), 2), rnd((D,), 3, torch.float32)
    y, mean, rstd = mx.layer_norm(x, w)
    dx, dw, _ = mx.layer_norm_backward(dy, x, w, mean, rstd)
    with checked():
        for call, want in ((lambda: mx.layer_norm(x, w)[0], y),
                           (lambda: mx.layer_norm_backward(dy, x, w, mean, rstd)[0], dx)):
            mx.mx_selftest_arm_stall(at)
            call()
            assert mx.mx_watchdog(clear=True) == 1
            assert torch.equal(call(), want)
            assert mx.mx_watchdog(clear=True) == 0
        assert mx.mx_bounds_check(clear=True) == 0


@pytest.mark.parametrize("M,D", [(6100, 1021), (330, 8190)])
def test_layer_norm_of_many_rows(M, D):
    test_layer_norm(M, D)


@pytest.mark.parametrize("M,N,K", [(2501, 1001, 160), (2501, 1002, 96), (300, 701, 160)])
def test_matmul_off_the_boundary(M, N, K):
    test_matmul(M, N, K)


def test_matmul_off_the_boundary_gives_up():
    a, b = mx.cast_dim0(rnd((2501, 1024), 1)), mx.cast_dim0(rnd((1001, 1024), 2))
    want = mx.matmul(*a, *b)
    with checked():
        mx.mx_selftest_arm_stall(5)
        mx.matmul(*a, *b)
        assert mx.mx_watchdog(clear=True) == 1
        assert torch.equal(mx.matmul(*a, *b), want)
        assert mx.mx_watchdog(clear=True) == 0
        assert mx.mx_bounds_check(clear=True) == 0
