"""Plain 64-bit forms of MX-FP4 and of the products joined with the gated SiLU, for the
tests: written from the definitions with torch, sharing no code with the library."""
import torch

from plain64 import F64, blocked_at, mx_values, scale_values

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def codes_of(q):
    """(R, C) e2m1 codes of packed bytes (R, C/2), the low half first."""
    return torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)


def e2m1_values(q):
    code = codes_of(q).to(torch.int64)
    grid = torch.tensor(GRID, dtype=F64, device=q.device)
    v = grid[code & 7]
    return torch.where(code >= 8, -v, v)


def mx4_values(q, s_blk):
    """What packed e2m1 bytes (R x C/2) with blocked scales stand for, in float64."""
    v = e2m1_values(q)
    R, C = v.shape
    s = scale_values(s_blk.reshape(-1)[blocked_at(R, C // 32, q.device)])
    return (v.reshape(R, C // 32, 32) * s[..., None]).reshape(R, C)


def values(q, s_blk, bits):
    return mx_values(q, s_blk) if bits == 8 else mx4_values(q, s_blk)


def cast_rows(x):
    """MX-FP4 cast of bf16 x (R x C) along rows: (packed bytes, blocked scales with zero
    padding).  The nearest of the eight magnitudes by comparing distances, of two equally
    near the one with the even code; magnitudes past 6 are 6."""
    R, C = x.shape
    v = x.to(F64).reshape(R, C // 32, 32)
    amax = v.abs().amax(-1)
    amax = torch.where(torch.isnan(v).any(-1), torch.full_like(amax, float("inf")), amax)
    finite = torch.isfinite(amax)
    e = torch.frexp(torch.where(finite, amax, torch.ones_like(amax)))[1].to(F64) - 1 - 2
    s = torch.where(amax == 0, torch.zeros_like(e), (e + 127).clamp(0, 254))
    a = (v * torch.exp2(127 - s)[..., None]).abs()
    a = torch.where(finite[..., None], a, torch.full_like(a, 6.0))
    grid = torch.tensor(GRID, dtype=F64, device=x.device)
    d = (a[..., None].clamp(max=6) - grid).abs()
    near = d == d.amin(-1, keepdim=True)
    even = torch.arange(8, device=x.device) % 2 == 0
    pick = near & (even | (near.sum(-1, keepdim=True) == 1))
    code = pick.to(torch.int64).argmax(-1)
    code = code + 8 * (torch.signbit(v) & finite[..., None])
    code = code.reshape(R, C // 2, 2).to(torch.uint8)
    q = code[..., 0] | (code[..., 1] << 4)
    s = torch.where(finite, s, torch.full_like(s, 255)).to(torch.uint8)
    blk = torch.zeros((R + 127) // 128 * ((C // 32 + 3) // 4) * 512, dtype=torch.uint8, device=x.device)
    blk[blocked_at(R, C // 32, x.device)] = s
    return q, blk


def product(a, b, bits):
    """(A B^T, sum |a b|) of two MX operands in float64, and the tolerance of a sum: an
    addition of one instruction's terms and the running sum cuts off at most a unit of the
    last of 24 bits of the largest magnitude that takes part, for each term and for the sum.
    """
    va, vb = values(*a, bits), values(*b, bits)
    steps = 32 if bits == 8 else 64
    size = va.abs() @ vb.abs().t()
    return va @ vb.t(), size, (va.shape[1] / steps + steps) * 2.0 ** -23 * size


# The hardware's exponential and reciprocal are off by a few units of 2^-22 each; with the
# fp32 operations around them well within:
FAST = 2.0 ** -18
BF16 = 2.0 ** -8
TINY = 2.0 ** -125


def swiglu_of(p, tol):
    """h of sums p = [g | u] that are off by at most tol, and how far a bf16 h may be off:
    silu's slope is below 1.1."""
    g, u = p.chunk(2, -1)
    tg, tu = tol.chunk(2, -1)
    act = g * torch.sigmoid(g)
    h = act * u
    off = 1.1 * tg * (u.abs() + tu) + act.abs() * tu + FAST * h.abs()
    return h, off * (1 + BF16) + BF16 * h.abs() + TINY


def swiglu_back_of(dh, tol, gu):
    """The gradient of [g | u] for dh off by at most tol, and how far a bf16 one may be."""
    g, u = gu.to(F64).chunk(2, -1)
    sg = torch.sigmoid(g)
    kg = sg * (1 + g * (1 - sg))
    size = sg * (1 + g.abs() * (1 - sg))
    dg, du = dh * u * kg, dh * g * sg
    out = torch.cat([dg, du], -1)
    off = torch.cat([tol * (u * kg).abs() + FAST * (dh * u).abs() * size,
                     tol * (g * sg).abs() + FAST * du.abs()], -1)
    return out, off * (1 + BF16) + BF16 * out.abs() + TINY
