"""Plain 64-bit forms of the training operators, for the tests: written from
the definitions with torch on the CPU or the GPU, sharing no code with the
library or the oracle."""
import torch

F64 = torch.float64


def e4m3_values(q):
    """e4m3 bytes (uint8) as float64, field by field; 0x7F and 0xFF are NaN."""
    b = q.to(torch.int64)
    ex, man = (b >> 3) & 15, (b & 7).to(F64)
    mag = torch.where(ex == 0, man / 512, (1 + man / 8) * torch.exp2(ex.to(F64) - 7))
    mag = torch.where((b & 127) == 127, torch.full_like(mag, float("nan")), mag)
    return torch.where(b >= 128, -mag, mag)


def blocked_at(R, C, device):
    """Byte of scale (r, c) in the 128x4 blocked layout of an R x C matrix."""
    r = torch.arange(R, device=device)[:, None]
    c = torch.arange(C, device=device)[None, :]
    return ((r // 128) * ((C + 3) // 4) + c // 4) * 512 + (r % 32) * 16 \
        + (r % 128) // 32 * 4 + c % 4


def scale_values(s):
    """e8m0 bytes as float64; 0xFF is NaN."""
    v = torch.exp2(s.to(F64) - 127)
    return torch.where(s == 255, torch.full_like(v, float("nan")), v)


def mx_values(q, s_blk):
    """What e4m3 bytes (R x C) with blocked scales stand for, in float64."""
    R, C = q.shape
    s = scale_values(s_blk.reshape(-1)[blocked_at(R, C // 32, q.device)])
    return (e4m3_values(q).reshape(R, C // 32, 32) * s[..., None]).reshape(R, C)


def layer_norm(x, w, b, eps):
    """(y, mean, rstd) in float64."""
    x = x.to(F64)
    mean = x.mean(-1)
    rstd = ((x - mean[:, None]).square().mean(-1) + eps) ** -0.5
    y = (x - mean[:, None]) * rstd[:, None] * w.to(F64)
    return (y if b is None else y + b.to(F64)), mean, rstd


def layer_norm_backward(dy, x, w, mean, rstd):
    """(dx, dw, db) in float64, and the sums of magnitudes that bound the
    rounding errors of each."""
    dy, x, w = dy.to(F64), x.to(F64), w.to(F64)
    mean, rstd = mean.to(F64)[:, None], rstd.to(F64)[:, None]
    xh = (x - mean) * rstd
    g = dy * w
    c1, c2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    dx = rstd * (g - c1 - xh * c2)
    size = rstd * (g.abs() + g.abs().mean(-1, keepdim=True)
                   + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
    return (dx, (dy * xh).sum(0), dy.sum(0)), (size, (dy * xh).abs().sum(0), dy.abs().sum(0))


def swiglu(gu):
    g, u = gu.to(F64).chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def swiglu_backward(dh, gu):
    g, u = gu.to(F64).chunk(2, -1)
    dh = dh.to(F64)
    sg = 1 / (1 + torch.exp(-g))
    return torch.cat([dh * u * sg * (1 + g * (1 - sg)), dh * g * sg], -1)
