"""The joined products at gates where the sigmoid leaves fp32's normal range (from -80 down
the kernels correct for it), with other factors so large that the results do not: forward,
and backward from either form of the saved values, of 8 bits above all, where a block's
scale byte decides whether its gates are corrected.

Tolerance: as in test_gpu_swiglu_gates.py, (16 + 2 |g|) 2^-23 of a result's terms, half a
unit in the last place of bf16, and what the sums may be off, carried through the formulas.
"""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from plain64 import F64, blocked_at, mx_values
from plain_fp4 import BF16, TINY, product, values
from test_gpu_matmul_swiglu import check_saved, off, operand

pytestmark = pytest.mark.gpu

BITS = [8, 4]
# Single tiles and CTA pairs; widths of whole and of partial tiles.
SIZES = [(9, 96), (300, 160), (1031, 2720), (2304, 2304)]


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()
    assert mx.mx_watchdog(clear=True) == 0
    yield
    torch.cuda.synchronize()
    assert mx.mx_watchdog(clear=True) == 0


def gates(M, F, seed):
    """Gates of four kinds of blocks of 32, neighbours unlike along rows and columns:
    ordinary; the largest just under 56 (saved with scale byte 124, no gate low); some of
    [-112, -81] (125); some of [-120, -81] and one of -128 (126)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn(M, F // 32, 32, generator=g, device="cuda").clamp(-4, 4)
    kind = (torch.arange(M, device="cuda")[:, None] + torch.arange(F // 32, device="cuda")) % 4
    some = torch.rand(v.shape, generator=g, device="cuda") < 0.3
    some[..., 5] = True
    share = torch.rand(v.shape, generator=g, device="cuda")
    for k, lo, hi, most in ((1, -54, -33, -55), (2, -112, -81, -104), (3, -120, -81, -128)):
        low = torch.where(some, lo + (hi - lo) * share, v)
        low[..., 17] = most
        v = torch.where((kind == k)[..., None], low, v)
    return v.reshape(M, F), kind


def swiglu_back_low(dh, tol, gu):
    """The gradient of [g | u] in 64 bits and how far a bf16 one may be."""
    g, u = gu.to(F64).chunk(2, -1)
    sg = torch.sigmoid(g)
    kg = sg * (1 + g * (1 - sg))
    e = (16 + 2 * g.abs()) * 2.0 ** -23
    size = sg * (1 + g.abs() * (1 - sg))
    dg, du = dh * u * kg, dh * g * sg
    room = torch.cat([tol * (u * kg).abs() + e * (dh * u).abs() * size, tol * (g * sg).abs() + e * du.abs()], -1)
    want = torch.cat([dg, du], -1)
    return want, room * (1 + BF16) + BF16 * want.abs() + TINY


@pytest.mark.parametrize("saved", [8, 16])
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,F", SIZES)
def test_backward(M, F, bits, saved):
    K = 128
    dy, w = operand(M, K, bits, M, 1e20), operand(F, K, bits, F, K ** -0.5)
    g, kind = gates(M, F, M + F)
    r = torch.Generator(device="cuda").manual_seed(M)
    gu = torch.cat([g, 1.5 * torch.randn(M, F, generator=r, device="cuda")], 1).to(torch.bfloat16)
    if saved == 8:
        q, s = mx.cast_dim0(gu)
        at = blocked_at(M, 2 * F // 32, "cuda")
        for k, byte in ((1, 124), (2, 125), (3, 126)):
            assert bool((s[at][:, :F // 32][kind == k] == byte).all())
        padded = torch.full_like(s, 255)
        padded[at] = s[at]
        got = mx.matmul_swiglu_backward(*dy, *w, (q, padded), bits=bits)
        gu = mx_values(q, padded)
    else:
        got = mx.matmul_swiglu_backward(*dy, *w, gu, bits=bits)
    dh, _, tol = product(dy, w, bits)
    want, room = swiglu_back_low(dh, tol, gu)
    # Low gates that count: far above what may be flushed, and lost if taken for others.
    counts = (gu[:, :F].double() < -80) & (want[:, F:].abs() > 2.0 ** 16 * TINY)
    for k in (2, 3):
        assert int((counts.reshape(M, -1, 32) & (kind == k)[..., None]).sum()) > M * F // 50
    off(got, want, room)


def whole(R, K, bits, seed, lo, hi, first=4, scale=1.0):
    """An operand of whole numbers lo .. hi times a power of two, `first` (4 or -4) at the head
    of every block, which it holds exactly."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(lo, hi + 1, (R, K), generator=g, device="cuda").float()
    x[:, ::32] = first
    x = (x * scale).to(torch.bfloat16)
    a = mx.cast_dim0(x) if bits == 8 else mx.cast_fp4_dim0(x)
    assert torch.equal(values(*a, bits), x.double())
    return a


@pytest.mark.parametrize("save", [False, True], ids=["plain", "save"])
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,F", SIZES)
def test_forward(M, F, bits, save):
    """Whole numbers: sums of 64 products of at most 16 are exact.  Ups near 2^90; gates about
    -47, with a deviation of 43."""
    K = 64
    x, gate = whole(M, K, bits, 1, -3, 4), whole(F, K, bits, 2, -4, 3, first=-4)
    up = whole(F, K, bits, 3, -3, 4, scale=2.0 ** 90)
    g, u = (values(*x, bits) @ values(*w, bits).t() for w in (gate, up))
    want = g * torch.sigmoid(g) * u
    room = (16 + 2 * g.abs()) * 2.0 ** -23 * want.abs()
    room = room * (1 + BF16) + BF16 * want.abs() + TINY
    assert int(((g < -81) & (want.abs() > 2.0 ** 16 * TINY)).sum()) > M * F // 50
    w = tuple(zip(gate, up))
    if save:
        h, q, s = mx.matmul_swiglu(*x, *w, save=True, bits=bits)
        p = torch.cat([g, u], 1)
        check_saved(q, s, p, torch.zeros_like(p))
    else:
        h = mx.matmul_swiglu(*x, *w, bits=bits)
    off(h, want, room)
