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
