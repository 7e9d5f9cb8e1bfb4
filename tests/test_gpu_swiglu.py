"""Gated SiLU, forward and backward, on the GPU against 64 bits.

Tolerance, fixed by the arithmetic: the exponential's documented error is
2 + 1.173 |g| units of 2^-23 and the division's 2, a handful of products follow:
(16 + 2 |g|) 2^-23 of each result's terms; a bf16 result adds 2^-8 of its value
(half a unit in the last place).  Below g = -87 the sigmoid, under 2^-125, may
come out as 0.
"""
import numpy as np
import pytest
import torch

import oracle
import mxfp8_block_scaled_dim0_gb300 as mx
import plain64
from mxfp8_block_scaled_dim0_gb300 import workloads as W

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
GUARD = 256


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()


def rnd(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF)


def guarded(shape, dtype):
    n = int(np.prod(shape))
    buf = torch.full((n + GUARD,), 9, dtype=dtype, device="cuda")
    return buf[:n].view(shape), buf[n:]


def forward(gu, save):
    M, F2 = gu.shape
    outs = [guarded((M, F2 // 2), BF)]
    if save:
        outs += [guarded((M, F2), torch.uint8),
                 guarded((mx.mx_blocked_bytes(M, F2 // 32),), torch.uint8)]
    mx.mx_swiglu(gu, *[t for t, _ in outs])
    torch.cuda.synchronize()
    for _, rest in outs:
        assert bool((rest == 9).all()), "written past the end"
    return [t for t, _ in outs]


def backward(dh, gu, saved):
    M, F = dh.shape
    out, rest = guarded((M, 2 * F), BF)
    q, s = saved if saved else (None, None)
    mx.mx_swiglu_backward(dh, gu, q, s, out)
    torch.cuda.synchronize()
    assert bool((rest == 9).all()), "written past the end"
    return out


def check_forward(gu, h):
    want = plain64.swiglu(gu)
    g, u = gu.double().chunk(2, -1)
    tol = want.abs() * (2.0 ** -8 + (16 + 2 * g.abs()) * 2.0 ** -23) + (g * u).abs() * 2.0 ** -125 \
        + 2.0 ** -133
    assert bool(((h.double() - want).abs() <= tol).all())


def check_backward(dh, gu, got):
    want = plain64.swiglu_backward(dh, gu)
    g, u = gu.double().chunk(2, -1)
    d, sg = dh.double().abs(), torch.sigmoid(g)
    e = (16 + 2 * g.abs()) * 2.0 ** -23
    tg = (d * u.abs() * sg * (1 + g.abs())) * e + d * u.abs() * (1 + g.abs()) * 2.0 ** -125
    tu = (d * g.abs() * sg) * e + d * g.abs() * 2.0 ** -125
    tol = torch.cat([tg, tu], -1) * (1 + 2.0 ** -7) + 2.0 ** -8 * want.abs() + 2.0 ** -133
    assert bool(((got.double() - want).abs() <= tol).all())


SHAPES = [(1, 1), (3, 5), (1, 7), (2, 62), (33, 250), (515, 2731), (5, 4102), (1, 8), (9, 40),
          (1, 32), (130, 32), (129, 96), (64, 128), (31, 160), (257, 224), (3, 4096), (1, 16384),
          (300, 1056)]


@pytest.mark.parametrize("M,F", SHAPES)
def test_forward_and_backward(M, F):
    gu, dh = rnd((M, 2 * F), M + F, 3.0), rnd((M, F), M + F + 1)
    check_forward(gu, forward(gu, False)[0])
    check_backward(dh, gu, backward(dh, gu, None))


# Rows a warp each, and from about 3000 128 x 128 tiles on a tile at a time.
@pytest.mark.parametrize("M,F", [s for s in SHAPES if s[1] % 32 == 0] + [(12501, 4096), (24900, 2048)])
def test_saved_input(M, F):
    if M * F <= 2000000:
        gu = W.spiky(M, 2 * F, M + F, scale_frac=0.05, zero_frac=0.05).cuda().clamp(-80, 80)
    else:
        gu = rnd((M, 2 * F), M + F, 3.0)
    dh = rnd((M, F), M + F + 1)
    h, q, s = forward(gu, True)
    assert torch.equal(h, forward(gu, False)[0])
    q0, s0 = mx.cast_dim0(gu)
    assert torch.equal(q, q0) and torch.equal(s, s0)
    if M * F <= 100000:
        oq, os_ = oracle.cast_dim0(W.bf16_bits(gu.cpu()))
        assert np.array_equal(q.cpu().numpy().ravel(), np.asarray(oq).ravel())
        assert np.array_equal(s.cpu().numpy().ravel(), np.asarray(oracle.to_blocked(os_)).ravel())
    check_backward(dh, plain64.mx_values(q, s), backward(dh, None, (q, s)))


def test_every_gate():
    """All finite bf16 gates, both ends included."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16)
    g = bits.view(BF)
    g = torch.where(torch.isfinite(g), g, torch.zeros_like(g)).view(64, 1024)
    gu = torch.cat([g, torch.full_like(g, 0.75)], 1)
    dh = torch.full_like(g, -1.5)
    small = g.double().abs() < 1e37                  # beyond, the product leaves bf16
    h = forward(gu, False)[0]
    want = plain64.swiglu(gu)
    tol = want.abs() * (2.0 ** -8 + (16 + 2 * g.double().abs().clamp(max=200)) * 2.0 ** -23) \
        + g.double().abs() * 2.0 ** -125 + 2.0 ** -133
    assert bool(((h.double() - want).abs() <= tol)[small].all())
    d = backward(dh, gu, None)
    assert bool(torch.isfinite(d[:, :1024][small]).all())
    want = plain64.swiglu_backward(dh, gu)
    ok = small & (g.double().abs() < 80)
    e = (16 + 2 * g.double().abs()) * 2.0 ** -23 * (1 + g.double().abs()) * 1.5
    both = (d.double() - want).abs() - 2.0 ** -8 * want.abs() - 2.0 ** -133
    assert bool((both[:, :1024][ok] <= e[ok]).all()) and bool((both[:, 1024:][ok] <= e[ok]).all())


def test_inf_and_nan_stay_where_they_are():
    gu, dh = rnd((4, 256), 1), rnd((4, 128), 2)
    gu[1, 3], gu[2, 130], gu[0, 7] = float("nan"), float("nan"), float("inf")
    h, q, s = forward(gu, True)
    nan = torch.isnan(h)
    assert bool(nan[1, 3]) and bool(nan[2, 2]) and int(nan.sum()) == 2
    assert bool(torch.isinf(h[0, 7]))
    q0, s0 = mx.cast_dim0(gu)
    assert torch.equal(q, q0) and torch.equal(s, s0)
    d = torch.isnan(backward(dh, gu, None))
    # u NaN spoils dg alone, g NaN both; g = inf gives inf * 0 in dg
    want = torch.zeros_like(d)
    want[1, 3] = want[1, 131] = want[2, 2] = want[0, 7] = True
    assert torch.equal(d, want)


def test_backward_against_differences():
    M, F, h = 16, 96, 1e-4
    gu, dh = rnd((M, 2 * F), 1, 2.0), rnd((M, F), 2)
    got = mx.swiglu_backward(dh, gu).double()
    g = torch.Generator(device="cuda").manual_seed(3)
    v = torch.randn((M, 2 * F), generator=g, device="cuda", dtype=torch.float64)
    f = lambda t: float((plain64.swiglu(t) * dh.double()).sum())  # noqa: E731
    want = (f(gu.double() + h * v) - f(gu.double() - h * v)) / (2 * h)
    tol = 4 * 2.0 ** -8 * float((got * v).square().sum().sqrt()) + 1e-3
    assert abs(float((got * v).sum()) - want) <= tol


def test_on_another_stream():
    gu, dh = rnd((700, 1024), 1), rnd((700, 512), 2)
    want, back = mx.swiglu(gu, save=True), mx.swiglu_backward(dh, gu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, gb = mx.swiglu(gu, save=True, stream=s), mx.swiglu_backward(dh, gu, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(gb, back)


def test_rows_beyond_32_bit_offsets():
    M, F = 70100, 16384
    gu = torch.empty((M, 2 * F), dtype=BF, device="cuda")
    gu[:] = rnd((1, 2 * F), 1)
    gu[M - 1] = rnd((2 * F,), 2)
    h, q, s = mx.swiglu(gu, save=True)
    check_forward(gu[M - 1:], h[M - 1:])
    assert torch.equal(h[M - 2], h[0])
    tail = M // 128 * 128
    q1, s1 = mx.cast_dim0(gu[tail:].contiguous())
    assert torch.equal(q[tail:], q1) and torch.equal(s[tail * (F // 16):], s1)
    del h
    got = mx.swiglu_backward(gu[:, :F].contiguous(), (q, s))
    check_backward(gu[tail:, :F], plain64.mx_values(q[tail:].contiguous(), s[tail * (F // 16):]),
                   got[tail:])


def test_refusals():
    gu, dh = rnd((8, 128), 1), rnd((8, 64), 2)
    h = torch.empty_like(dh)
    with pytest.raises(ValueError, match="even"):
        mx.mx_swiglu(rnd((4, 33), 1), h)
    with pytest.raises(ValueError, match="h must have shape"):
        mx.mx_swiglu(gu, h[:4])
    with pytest.raises(TypeError, match="gu must"):
        mx.mx_swiglu(gu.float(), h)
    with pytest.raises(ValueError, match="contiguous"):
        mx.mx_swiglu(gu.t().contiguous().t(), h)
    with pytest.raises(ValueError, match="go together"):
        mx.mx_swiglu(gu, h, torch.empty(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="give gu, or"):
        mx.mx_swiglu_backward(dh, None, None, None, gu)
    with pytest.raises(ValueError, match="CUDA"):
        mx.mx_swiglu(gu, h.cpu())
    with pytest.raises(mx.MXError):
        mx.swiglu(rnd((2, 96), 1), save=True)        # 48 gates: no whole blocks
