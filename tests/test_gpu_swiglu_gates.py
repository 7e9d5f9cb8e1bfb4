"""Gated SiLU at gates where the sigmoid leaves fp32's normal range (below -87.3)
while its products with ordinary numbers do not, against 64 bits.

Tolerance, as for other gates: (16 + 2 |g|) 2^-23 of a result's terms and half a
unit in the last place of bf16, here without an allowance for sigmoids under
2^-126; results under bf16's normal range to half its smallest number.  exp(g) is
reached as the square of exp(g / 2), whose own last bits are lost below g = -174.7
(under fp32's normal range): 2^-7 there.
"""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
import plain64

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()


def gates(F):
    """Every bf16 gate of [-210, -60], and ordinary ones, each with u and dh of
    many sizes: rows of F gates."""
    low = torch.arange(0xC270, 0xC353, device="cuda").to(torch.int32)
    g = (low << 16).view(torch.float32)
    g = torch.cat([g, torch.linspace(-60, 60, 60, device="cuda")]).to(BF)
    u = torch.tensor([1.0, -0.75, 3e-5, 7e8, -2e17, 1.5e27, -3e37], device="cuda").to(BF)
    d = torch.tensor([1.0, -0.5, 4e-6, 3.0], device="cuda").to(BF)      # d u within fp32
    g, u, d = (t.reshape(-1) for t in torch.meshgrid(g, u, d, indexing="ij"))
    pad = -len(g) % F
    g, u, d = (torch.cat([t, torch.ones(pad, dtype=BF, device="cuda")]).view(-1, F) for t in (g, u, d))
    return g, u, d


def close(got, want, g, terms):
    e = (16 + 2 * g.abs()) * 2.0 ** -23 + torch.where(g < -174.7, 2.0 ** -7, 0.0)
    tol = terms.abs() * e * (1 + 2.0 ** -7) + 2.0 ** -8 * want.abs() + 2.0 ** -133
    fits = want.abs() < 1e38                         # what bf16 can hold
    bad = fits & ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), (g[bad], want[bad], got[bad])


@pytest.mark.parametrize("F", [1, 62, 96, 128, 250, 1024])
def test_low_gates(F):
    g, u, d = gates(F)
    gu = torch.cat([g, u], 1).contiguous()
    gd, ud, dd = g.double(), u.double(), d.double()
    want = plain64.swiglu(gu)
    close(mx.swiglu(gu), want, gd, want)
    got = mx.swiglu_backward(d, gu)
    wg, wu = plain64.swiglu_backward(d, gu).chunk(2, -1)
    close(got[:, :F], wg, gd, wg)
    close(got[:, F:], wu, gd, wu)


@pytest.mark.parametrize("F", [96, 128, 1024])
def test_low_gates_saved(F):
    g, u, d = gates(F)
    gu = torch.cat([g, u], 1).contiguous()
    h, q, s = mx.swiglu(gu, save=True)
    assert torch.equal(h, mx.swiglu(gu))
    q0, s0 = mx.cast_dim0(torch.cat([gu, gu.new_zeros(-len(gu) % 32, 2 * F)]))
    assert torch.equal(q, q0[:len(gu)]) and torch.equal(s, s0)
    x = plain64.mx_values(q, s)
    got = mx.swiglu_backward(d, (q, s))
    wg, wu = plain64.swiglu_backward(d, x).chunk(2, -1)
    close(got[:, :F], wg, x[:, :F], wg)
    close(got[:, F:], wu, x[:, :F], wu)


@pytest.mark.parametrize("M,F", [(16001, 251), (16001, 250), (16001, 264), (16001, 288), (12501, 4096)])
def test_few_low_gates_among_many(M, F):
    """A thread's many pieces, one gate in a few thousand low; the tiles' kernel too."""
    r = torch.Generator(device="cuda").manual_seed(M + F)
    gu = 3 * torch.randn((M, 2 * F), generator=r, device="cuda")
    low = torch.rand((M, F), generator=r, device="cuda") < 3e-4
    gu[:, :F] = torch.where(low, -80 - 60 * torch.rand((M, F), generator=r, device="cuda"), gu[:, :F])
    gu[:, F:] = torch.where(low, gu[:, F:] * 1e30, gu[:, F:])
    gu = gu.to(BF)
    d = torch.randn((M, F), generator=r, device="cuda").to(BF)
    h, back = mx.swiglu(gu), mx.swiglu_backward(d, gu)
    rows = torch.cat([torch.arange(300), torch.arange(M // 2, M // 2 + 300), torch.arange(M - 300, M)]).cuda()
    gd = gu[rows, :F].double()
    assert bool((gd < -80).any())
    want = plain64.swiglu(gu[rows])
    close(h[rows], want, gd, want)
    wg, wu = plain64.swiglu_backward(d[rows], gu[rows]).chunk(2, -1)
    close(back[rows, :F], wg, gd, wg * (1 + gd.abs()))
    close(back[rows, F:], wu, gd, wu)
    if F % 32 == 0:
        hs, q, s = mx.swiglu(gu, save=True)
        assert torch.equal(hs, h)


def test_infinite_gates():
    """exp(-inf) is 0 and 0 times infinity no number, as the formula has it."""
    for F in (1, 2, 8, 128):
        gu = torch.ones((3, 2 * F), device="cuda")
        gu[0, 0], gu[1, 0], gu[2, 0] = float("-inf"), float("inf"), float("nan")
        gu = gu.to(BF)
        h = mx.swiglu(gu)
        assert bool(torch.isnan(h[0, 0])) and float(h[1, 0]) == float("inf") and bool(torch.isnan(h[2, 0]))
        assert bool(torch.isfinite(h[:, 1:]).all())
        d = mx.swiglu_backward(torch.ones((3, F), device="cuda").to(BF), gu)
        assert bool(torch.isnan(d[0, 0])) and bool(torch.isnan(d[0, F])) and float(d[1, F]) == float("inf")
