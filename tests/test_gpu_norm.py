"""Layer norm, forward and backward, on the GPU against 64 bits.

Tolerances, fixed by the arithmetic.  A sum over a row goes through at most 16
additions in a thread, then two trees of five: every partial sum is rounded to
24 bits, so a mean is within 32 2^-24 of the mean magnitude.  rstd follows from
deviations that are off by the mean's error, which only counts squared, and by
their own rounding: 64 2^-24 of it.  Results in bf16 add half a unit in the last
place, 2^-8 of the value.  Sums over M rows take at most M + 64 additions.
"""
import numpy as np
import pytest
import torch

import oracle
import mxfp8_block_scaled_dim0_gb300 as mx
import plain64
from mxfp8_block_scaled_dim0_gb300 import workloads as W

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
BF, F32 = torch.bfloat16, torch.float32
GUARD = 256


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()


def rnd(shape, seed, dtype=BF, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


def guarded(shape, dtype):
    n = int(np.prod(shape))
    buf = torch.full((n + GUARD,), 9, dtype=dtype, device="cuda")
    return buf[:n].view(shape), buf[n:]


def forward(x, w, b, save, eps=EPS):
    M, D = x.shape
    outs = [guarded((M, D), BF), guarded((M,), F32), guarded((M,), F32)]
    if save:
        outs += [guarded((M, D), torch.uint8),
                 guarded((mx.mx_blocked_bytes(M, D // 32),), torch.uint8)]
    mx.mx_layer_norm(x, w, b, eps, *[t for t, _ in outs])
    torch.cuda.synchronize()
    for _, rest in outs:
        assert bool((rest == 9).all()), "written past the end"
    return [t for t, _ in outs]


def check_forward(x, w, b, got, eps=EPS):
    y, mean, rstd = got[:3]
    y64, m64, r64 = plain64.layer_norm(x, w, b, eps)
    off = 32 * U * x.double().abs().mean(-1)
    assert bool(((mean.double() - m64).abs() <= off).all())
    rel = 64 * U + (off * r64) ** 2
    assert bool(((rstd.double() - r64).abs() <= rel * r64).all())
    wd = w.double().abs()
    xh = (y64 if b is None else y64 - b.double()).abs()
    tol = 2.0 ** -8 * y64.abs() + xh * (rel + 8 * U)[:, None] + (off * r64)[:, None] * wd \
        + (0 if b is None else 4 * U * b.double().abs())
    assert bool(((y.double() - y64).abs() <= tol * (1 + 2.0 ** -7)).all())


ODD = [(1, 1), (2, 3), (9, 1), (1300, 5), (2500, 12), (1219, 250), (640, 514), (165, 1020), (1, 7), (5, 31), (3, 130), (33, 257), (7, 1021), (9, 1022), (4, 4099),
       (2, 16383), (3, 16382)]
EVEN = [(1, 32), (1, 4096), (129, 96), (31, 160), (300, 512), (5, 544), (130, 1024), (65, 1056),
        (40, 5120), (17, 8192), (3, 16384), (700, 64), (9, 16360)]


@pytest.mark.parametrize("wt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D", ODD + EVEN)
def test_forward(M, D, wt):
    x = rnd((M, D), M + D, scale=2.0, shift=0.5)
    w, b = rnd((D,), 1, wt, 0.2, 1.0), rnd((D,), 2, wt, 0.3)
    check_forward(x, w, b, forward(x, w, b, False))
    check_forward(x, w, None, forward(x, w, None, False))


@pytest.mark.parametrize("wt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D", [s for s in EVEN if s[1] % 32 == 0])
def test_forward_saves_the_dim0_cast(M, D, wt):
    x = W.spiky(M, D, M + D, scale_frac=0.05, zero_frac=0.05).cuda()
    x[0] = x[0] + 1
    w, b = rnd((D,), 1, wt, 0.2, 1.0), rnd((D,), 2, wt, 0.3)
    got = forward(x, w, b, True)
    plain = forward(x, w, b, False)
    for a, c in zip(got[:3], plain):
        assert torch.equal(a, c)
    q0, s0 = mx.cast_dim0(x)
    assert torch.equal(got[3], q0) and torch.equal(got[4], s0)
    if M * D <= 200000:
        oq, os_ = oracle.cast_dim0(W.bf16_bits(x.cpu()))
        assert np.array_equal(got[3].cpu().numpy().ravel(), np.asarray(oq).ravel())
        assert np.array_equal(got[4].cpu().numpy().ravel(), np.asarray(oracle.to_blocked(os_)).ravel())


def test_large_mean_small_spread():
    """Deviations far below the mean: the two-pass variance keeps them."""
    x = rnd((64, 2048), 5, scale=0.5, shift=64.0)
    w, b = rnd((2048,), 1, F32, 0.2, 1.0), rnd((2048,), 2, F32)
    check_forward(x, w, b, forward(x, w, b, False))


def test_constant_rows_and_eps():
    x = torch.full((3, 96), 2.0, dtype=BF, device="cuda")
    w, b = rnd((96,), 1, F32), rnd((96,), 2, F32)
    y, mean, rstd = forward(x, w, b, False, eps=1e-2)
    assert bool((mean == 2).all()) and bool(((rstd - 10).abs() <= 10 * 4 * 2 * U).all())
    assert torch.equal(y, b.to(BF).expand(3, 96))
    y, _, rstd = forward(x, w, b, False, eps=0.0)      # 0 / 0: NaN, as the formula has it
    assert bool(torch.isinf(rstd).all()) and bool(torch.isnan(y).all())


def test_inf_and_nan_stay_in_their_rows():
    x = rnd((6, 640), 3)
    x[1, 5], x[3, 639], x[4, 0] = float("inf"), float("nan"), -float("inf")
    w, b = rnd((640,), 1, F32), rnd((640,), 2, F32)
    y, mean, rstd, q, s = forward(x, w, b, True)
    bad = torch.tensor([1, 3, 4], device="cuda")
    good = torch.tensor([0, 2, 5], device="cuda")
    assert bool(torch.isnan(y[bad]).all()) and bool(torch.isnan(rstd[bad]).all())
    check_forward(x[good], w, b, (y[good], mean[good], rstd[good]))
    q0, s0 = mx.cast_dim0(x)
    assert torch.equal(q, q0) and torch.equal(s, s0)


@pytest.mark.parametrize("D", [1, 13, 127, 254, 637, 1028, 4100])
def test_neighbours_of_rows_off_the_boundary(D):
    """Rows that do not begin on 16 bytes: what a copy brings of a row's
    neighbours, NaN here, reaches neither its results nor theirs."""
    M = 40
    x, dy = rnd((M, D), 3, shift=1.0), rnd((M, D), 4)
    w, b = rnd((D,), 1, F32), rnd((D,), 2, F32)
    mean, rstd = stats(x)
    xn, dyn, mn, rn = x.clone(), dy.clone(), mean.clone(), rstd.clone()
    xn[1::2], dyn[1::2], mn[1::2], rn[1::2] = (float("nan"),) * 4
    y = forward(xn, w, b, False)[0]
    assert bool(torch.isnan(y[1::2]).all())
    assert torch.equal(y[::2], forward(x, w, b, False)[0][::2])
    dx = backward(dyn, xn, None, w, mn, rn)[0]
    assert bool(torch.isnan(dx[1::2]).all())
    assert torch.equal(dx[::2], backward(dy, x, None, w, mean, rstd)[0][::2])


# ---- backward ------------------------------------------------------------------

def backward(dy, x, saved, w, mean, rstd, bias=True):
    M, D = dy.shape
    outs = [guarded((M, D), BF), guarded((D,), w.dtype), guarded((D,), w.dtype)]
    work, rest = guarded((mx.mx_layer_norm_backward_work_bytes(M, D),), torch.uint8)
    q, s = saved if saved else (None, None)
    mx.mx_layer_norm_backward(dy, x, q, s, w, mean, rstd, outs[0][0], outs[1][0],
                              outs[2][0] if bias else None, work)
    torch.cuda.synchronize()
    assert bool((rest == 9).all()), "scratch written past its end"
    for _, rest in outs:
        assert bool((rest == 9).all()), "written past the end"
    return [t for t, _ in outs]


def check_backward(dy, x, w, mean, rstd, got):
    M = dy.shape[0]
    want, size = plain64.layer_norm_backward(dy, x, w, mean, rstd)
    n = [48 * U, (M + 64) * U, (M + 64) * U]
    for k, name in enumerate(("dx", "dw", "db")):
        tol = n[k] * size[k]
        if got[k].dtype == BF:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want[k].abs() + 2.0 ** -133
        off = (got[k].double() - want[k]).abs()
        assert bool((off <= tol).all()), "%s: %g" % (name, float((off - tol).max()))


def stats(x):
    _, mean, rstd = plain64.layer_norm(x, torch.ones(x.shape[1], device="cuda"), None, EPS)
    return mean.float(), rstd.float()


@pytest.mark.parametrize("wt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D", ODD + EVEN + [(1031, 1021), (2000, 264), (1500, 96)])
def test_backward(M, D, wt):
    x, dy = rnd((M, D), M + D, scale=2.0, shift=0.5), rnd((M, D), M + D + 1, scale=1e-2)
    w = rnd((D,), 1, wt, 0.2, 1.0)
    mean, rstd = stats(x)
    check_backward(dy, x, w, mean, rstd, backward(dy, x, None, w, mean, rstd))


@pytest.mark.parametrize("wt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D", [s for s in EVEN if s[1] % 32 == 0] + [(2000, 288)])
def test_backward_from_the_saved_input(M, D, wt):
    x, dy = rnd((M, D), M + D, scale=2.0, shift=0.5), rnd((M, D), M + D + 1, scale=1e-2)
    w = rnd((D,), 1, wt, 0.2, 1.0)
    y, mean, rstd, q, s = mx.layer_norm(x, w, None, EPS, save=True)
    got = backward(dy, None, (q, s), w, mean, rstd)
    check_backward(dy, plain64.mx_values(q, s), w, mean, rstd, got)


def test_backward_without_bias_gradient():
    x, dy = rnd((70, 200), 1), rnd((70, 200), 2)
    w = rnd((200,), 3, F32)
    mean, rstd = stats(x)
    dx, dw, db = backward(dy, x, None, w, mean, rstd)
    dx2, dw2, db2 = backward(dy, x, None, w, mean, rstd, bias=False)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and bool((db2 == 9).all())


def test_backward_of_every_saved_byte():
    """All 256 element bytes under all scales that occur: what a save of any
    bf16 row can hold."""
    q = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(256, 1)
    q[(q & 127) == 127] = 0
    s = torch.zeros(mx.mx_blocked_bytes(256, 8), dtype=torch.uint8, device="cuda")
    s[plain64.blocked_at(256, 8, "cuda")] = torch.arange(256, device="cuda").clamp(max=247).to(torch.uint8)[:, None]
    x = plain64.mx_values(q, s)
    _, mean, rstd = plain64.layer_norm(x, torch.ones(256, device="cuda"), None, 1e-30)
    mean, rstd = mean.float(), rstd.float()
    dy = rnd((256, 256), 5)
    w = torch.ones(256, device="cuda")
    # Rows whose squares or reciprocals leave fp32 have no such answer.
    r = (s[plain64.blocked_at(256, 8, "cuda")][:, 0] > 80) & (s[plain64.blocked_at(256, 8, "cuda")][:, 0] < 180)
    dx, _, _ = backward(dy, None, (q, s), w, mean, rstd)
    want, size = plain64.layer_norm_backward(dy[r], x[r], w, mean[r], rstd[r])
    assert bool(((dx[r].double() - want[0]).abs() <= 2.0 ** -8 * want[0].abs() + 64 * U * size[0]).all())


def test_backward_against_differences():
    """<dx, v> and <dw, t> of the GPU against differences of the 64-bit forward
    pass."""
    M, D, h = 24, 352, 1e-4
    x, dy = rnd((M, D), 1), rnd((M, D), 2)
    w, b = rnd((D,), 3, F32, 0.2, 1.0), rnd((D,), 4, F32)
    _, mean, rstd = mx.layer_norm(x, w, b, EPS)
    dx, dw, db = mx.layer_norm_backward(dy, x, w, mean, rstd)

    def loss(x, w, b):
        return float((plain64.layer_norm(x, w, b, EPS)[0] * dy.double()).sum())

    def differ(f, t, v):
        return (f(t.double() + h * v) - f(t.double() - h * v)) / (2 * h)

    v, t = rnd((M, D), 5, torch.float64), rnd((D,), 6, torch.float64)
    # dx: M D independent roundings to bf16 (2^-8 of each term, at random signs
    # their root sum of squares; four of these); the differences' own error h^2
    tol = 4 * 2.0 ** -8 * float((dx.double() * v).square().sum().sqrt()) + 1e-3
    assert abs(float((dx.double() * v).sum()) - differ(lambda a: loss(a, w, b), x, v)) <= tol
    assert abs(float((dw.double() * t).sum()) - differ(lambda a: loss(x, a, b), w, t)) <= 2e-3
    assert abs(float((db.double() * t).sum()) - differ(lambda a: loss(x, w, a), b, t)) <= 2e-3


@pytest.mark.parametrize("M,D", [(3000, 96), (1500, 1021), (700, 4096)])
def test_backward_same_bits_every_time(M, D):
    x, dy, w = rnd((M, D), 1), rnd((M, D), 2), rnd((D,), 3, F32)
    mean, rstd = stats(x)
    first = mx.layer_norm_backward(dy, x, w, mean, rstd)
    for _ in range(3):
        for a, b in zip(mx.layer_norm_backward(dy, x, w, mean, rstd), first):
            assert torch.equal(a, b)


def test_on_another_stream():
    x, dy, w = rnd((900, 640), 1), rnd((900, 640), 2), rnd((640,), 3, F32)
    mean, rstd = stats(x)
    want = mx.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [mx.layer_norm_backward(dy, x, w, mean, rstd, stream=s) for _ in range(3)]
    raw = mx.layer_norm_backward(dy, x, w, mean, rstd, stream=s.cuda_stream)
    fwd = mx.layer_norm(x, w, None, EPS, save=True, stream=s)
    s.synchronize()
    for g in got + [raw]:
        for a, b in zip(g, want):
            assert torch.equal(a, b)
    for a, b in zip(fwd, mx.layer_norm(x, w, None, EPS, save=True)):
        assert torch.equal(a, b)


def test_rows_beyond_32_bit_offsets():
    """M D above 2^31 values."""
    M, D = 140000, 16384
    x = torch.empty((M, D), dtype=BF, device="cuda")
    x[:] = rnd((1, D), 1)
    x[M - 1] = rnd((D,), 2)
    w, b = rnd((D,), 3, F32), rnd((D,), 4, F32)
    y, mean, rstd, q, s = mx.layer_norm(x, w, b, EPS, save=True)
    check_forward(x[M - 1:], w, b, (y[M - 1:], mean[M - 1:], rstd[M - 1:]))
    assert torch.equal(y[M - 2], y[0])
    tail = M // 128 * 128
    q1, s1 = mx.cast_dim0(x[tail:].contiguous())
    assert torch.equal(q[tail:], q1) and torch.equal(s[tail * (D // 32):], s1)
    del y
    dx, dw, db = mx.layer_norm_backward(x, (q, s), w, mean, rstd)
    xv = plain64.mx_values(q[tail:].contiguous(), s[tail * (D // 32):])
    want, size = plain64.layer_norm_backward(x[tail:], xv, w, mean[tail:], rstd[tail:])
    assert bool(((dx[tail:].double() - want[0]).abs()
                 <= 2.0 ** -8 * want[0].abs() + 64 * U * size[0] + 2.0 ** -133).all())


def test_refusals():
    x, w = rnd((8, 64), 1), rnd((64,), 2, F32)
    y, m, r = torch.empty_like(x), torch.empty(8, device="cuda"), torch.empty(8, device="cuda")
    with pytest.raises(TypeError, match="x must"):
        mx.mx_layer_norm(x.half(), w, None, EPS, y, m, r)
    with pytest.raises(ValueError, match="w must have shape"):
        mx.mx_layer_norm(x, w[:32], None, EPS, y, m, r)
    with pytest.raises(TypeError, match="b must"):
        mx.mx_layer_norm(x, w, w.to(BF), EPS, y, m, r)
    with pytest.raises(ValueError, match="contiguous"):
        mx.mx_layer_norm(x.t().contiguous().t(), w, None, EPS, y, m, r)
    with pytest.raises(ValueError, match="go together"):
        mx.mx_layer_norm(x, w, None, EPS, y, m, r, torch.empty(512, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="give x, or"):
        mx.mx_layer_norm_backward(x, None, None, None, w, m, r, y, w, w, w)
    with pytest.raises(ValueError, match="work holds"):
        mx.mx_layer_norm_backward(x, x, None, None, w, m, r, y, w, w, w)
    with pytest.raises(mx.MXError):
        mx.layer_norm(rnd((2, 48), 1), rnd((48,), 1, F32), save=True)
    with pytest.raises(mx.MXError):
        mx.layer_norm(rnd((2, 16392), 1), rnd((16392,), 1, F32))


# Enough rows that each SM works through many, with every share of a row to a
# thread; lengths just past a multiple of 1024, and off the 16-byte boundary.
MANY = [(6100, 1021), (3100, 2050), (330, 8190), (2500, 4104), (6100, 1504), (1300, 5127),
        (10000, 640), (6100, 1361), (3100, 2296)]


@pytest.mark.parametrize("M,D", MANY)
def test_many_rows(M, D):
    x, dy = rnd((M, D), 3, scale=2.0, shift=0.5), rnd((M, D), 4, scale=1e-2)
    w, b = rnd((D,), 1, F32, 0.2, 1.0), rnd((D,), 2, F32, 0.3)
    check_forward(x, w, b, forward(x, w, b, False))
    mean, rstd = stats(x)
    check_backward(dy, x, w, mean, rstd, backward(dy, x, None, w, mean, rstd))


@pytest.mark.parametrize("M,D", [(2600, 5120), (330, 16384), (1300, 8224), (10001, 640), (6100, 1504),
                                 (3100, 2304)])
def test_many_saved_rows(M, D):
    x, dy = rnd((M, D), 3, scale=2.0, shift=0.5), rnd((M, D), 4, scale=1e-2)
    w = rnd((D,), 1, BF, 0.2, 1.0)
    y, mean, rstd, q, s = mx.layer_norm(x, w, None, EPS, save=True)
    got = backward(dy, None, (q, s), w, mean, rstd)
    check_backward(dy, plain64.mx_values(q, s), w, mean, rstd, got)


@pytest.mark.parametrize("M,D", [(6100, 1021), (330, 8190)])
def test_neighbours_among_many_rows(M, D):
    x, dy = rnd((M, D), 3, shift=1.0), rnd((M, D), 4)
    w, b = rnd((D,), 1, F32), rnd((D,), 2, F32)
    mean, rstd = stats(x)
    y, dx = forward(x, w, b, False)[0], backward(dy, x, None, w, mean, rstd)[0]
    x[1::2], dy[1::2], mean[1::2], rstd[1::2] = (float("nan"),) * 4
    assert torch.equal(forward(x, w, b, False)[0][::2], y[::2])
    assert torch.equal(backward(dy, x, None, w, mean, rstd)[0][::2], dx[::2])


@pytest.mark.parametrize("M", [1, 31, 32, 33, 97, 127, 129, 250])
def test_scales_of_rows_past_the_matrix(M):
    x, w = rnd((M, 416), M), rnd((416,), 1, F32)
    _, _, _, q, s = mx.layer_norm(x, w, save=True)
    q0, s0 = mx.cast_dim0(x.contiguous()) if M % 32 == 0 else (None, None)
    rows = (M + 127) // 128 * 128
    at = plain64.blocked_at(rows, 16, "cuda")
    assert bool((s[at[M:]] == 0).all()) and bool((s[at[:, 13:]] == 0).all())
    if s0 is not None:
        assert torch.equal(s, s0) and torch.equal(q, q0)
