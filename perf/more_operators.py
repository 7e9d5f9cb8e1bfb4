"""Measured cases of the operators that run a gated feed-forward layer on MX operands of
4 or 8 bits: the casts to MX-FP4 and back, the product of two MX-FP4 operands, and the
products that are joined with the gated SiLU, forward and backward.

``own`` false: every operator in plain form, elementary torch operations in 32 bits,
rounded once at the end.  ``own`` true: the framework's entry points.  ``exact``
computes the same results in 64 bits, from the definitions.

4-bit results come back as the packed bytes (two e2m1 codes, the first in the low half)
and scale bytes: whole numbers, equal bit for bit.
"""
import math

import torch

own = False

DEV = "cuda"


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # The activations of one token on their way into a 4-bit product: launch latency.
        dict(name="cast4 1x5120", op="cast", M=1, K=5120, dims="0"),
        # The MoE layer's activations for a training step, both directions in one read.
        dict(name="cast4 both 16640x5120", op="cast", M=16640, K=5120, dims="01"),
        # An expert's weights back in bf16.
        dict(name="dequant4 8192x5120", op="dequant", M=8192, K=5120),
        # Ragged rows of an odd width.
        dict(name="dequant4 515x2720", op="dequant", M=515, K=2720),
        # One token through the expert weights (8192 x 5120) while decoding.
        dict(name="product4 1x8192x5120", op="product", M=1, N=8192, K=5120, out="bf16"),
        # All tokens through them.
        dict(name="product4 16640x8192x5120", op="product", M=16640, N=8192, K=5120, out="bf16"),
        # The weight gradient of that layer: a long sum over the tokens, in fp32.
        dict(name="product4 8192x5120x16640", op="product", M=8192, N=5120, K=16640, out="f32"),
        # Gate and up projection of one token with 4-bit weights.
        dict(name="gated4 1x8192x5120", op="gated", M=1, F=8192, K=5120, bits=4, save=False),
        # The same layer's forward pass in training, gate and up saved in 8 bits.
        dict(name="gated8 save 16640x8192x5120", op="gated", M=16640, F=8192, K=5120, bits=8, save=True),
        # A ragged batch through a small layer of an odd width.
        dict(name="gated8 515x2720x1024", op="gated", M=515, F=2720, K=1024, bits=8, save=False),
        # Backward of the large layer: the gradient through the second product and the gate.
        dict(name="gated8 back 16640x8192x5120", op="gated_back", M=16640, F=8192, K=5120, bits=8, saved=8),
        # Backward of a micro-batch with 4-bit operands, gate and up kept in bf16.
        dict(name="gated4 back 1031x1376x1024", op="gated_back", M=1031, F=1376, K=1024, bits=4, saved=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _of(n, step):
    return max(step, n // step * step)


def draw(rng):
    op = rng.choice(["cast", "dequant", "product", "gated", "gated_back"])
    M = _log(rng, 1, 16640)
    if op in ("cast", "dequant"):
        K = _of(_log(rng, 32, 16384), 32)
        M = min(M, 16640 * 5120 // K)
        if op == "dequant":
            return dict(op=op, M=M, K=K)
        dims = rng.choice(["0", "1", "01"])
        return dict(op=op, M=M if dims == "0" else _of(M, 32), K=K, dims=dims)
    bits = rng.choice([4, 8])
    K = min(5120, _of(_log(rng, 64, 8192), 32 if bits == 8 and op != "product" else 64))
    if op == "product":
        return dict(op=op, M=M, N=_log(rng, 32, 8192), K=K, out=rng.choice(["bf16", "f32"]))
    F = _of(_log(rng, 32, 8192), 32)
    if op == "gated":
        return dict(op=op, M=M, F=F, K=K, bits=bits, save=rng.random() < 0.5)
    return dict(op=op, M=M, F=F, K=K, bits=bits, saved=rng.choice([8, 16]))


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "cast":
        return {"bytes": 2 * M * K + len(case["dims"]) * (M * K / 2 + M * K / 32), "flops": 4 * M * K}
    if op == "dequant":
        return {"bytes": M * K / 2 + M * K / 32 + 2 * M * K, "flops": 2 * M * K}
    if op == "product":
        N, size = case["N"], 2 if case["out"] == "bf16" else 4
        return {"bytes": (M + N) * K * 17 / 32 + size * M * N, "flops": 2 * M * N * K}
    F, a_value = case["F"], case["bits"] / 8 + 1 / 32
    if op == "gated":
        return {"bytes": (M + 2 * F) * K * a_value + 2 * M * F + (2 * M * F * 33 / 32 if case["save"] else 0),
                "flops": 4 * M * F * K + 8 * M * F}
    saved = 2 * M * F * (33 / 32 if case["saved"] == 8 else 2)
    return {"bytes": (M + F) * K * a_value + saved + 4 * M * F, "flops": 2 * M * F * K + 14 * M * F}


# ---- inputs --------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _hidden(g, M, D):
    """Activations: some loud channels, tokens of uneven size."""
    x = _randn(g, M, D).mul_(torch.exp(0.5 * _randn(g, 1, D)))
    return x.mul_(torch.exp(0.3 * _randn(g, M, 1))).to(torch.bfloat16)


def _weights(g, N, K):
    return _randn(g, N, K).mul_(1.2 * K ** -0.5).to(torch.bfloat16)


def _gradient(g, M, D):
    return _randn(g, M, D).mul_(1e-3 * torch.exp(0.5 * _randn(g, M, 1))).to(torch.bfloat16)


def _operand(x, bits):
    """(bytes, blocked scales) of x cast along its rows."""
    q, s = _cast8(x) if bits == 8 else _cast4(x)
    return q, _blocked(s)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, M, K = case["op"], case["M"], case["K"]
    st = dict(case=case)
    if op == "cast":
        st["x"] = _hidden(g, M, K)
    elif op == "dequant":
        st["a"] = _operand(_hidden(g, M, K), 4)
    elif op == "product":
        st["a"] = _operand(_hidden(g, M, K), 4)
        st["b"] = _operand(_weights(g, case["N"], K), 4)
    elif op == "gated":
        st["a"] = _operand(_hidden(g, M, K), case["bits"])
        st["gate"] = _operand(_weights(g, case["F"], K), case["bits"])
        st["up"] = _operand(_weights(g, case["F"], K), case["bits"])
    else:
        F = case["F"]
        st["a"] = _operand(_gradient(g, M, K), case["bits"])
        st["b"] = _operand(_weights(g, F, K), case["bits"])
        gu = (1.5 * _randn(g, M, 2 * F)).to(torch.bfloat16)
        st["saved"] = _operand(gu, 8) if case["saved"] == 8 else gu
    return st


# ---- plain forms ---------------------------------------------------------------

def _scaled(x, emax):
    """Blocks of 32 of x's rows, divided by their power of two, and the scale bytes."""
    R, C = x.shape
    v = x.float().reshape(R, C // 32, 32)
    e = v.abs().amax(-1).view(torch.int32) >> 23
    s = (e - emax).clamp(min=0)
    mult = ((254 - s) << 23).view(torch.float32)
    return v * mult[..., None], s.to(torch.uint8)


def _cast8(x):
    v, s = _scaled(x, 8)
    return v.clamp(-448, 448).to(torch.float8_e4m3fn).reshape(x.shape).view(torch.uint8), s


def _cast4(x):
    """e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), ties to the even code, two a byte."""
    v, s = _scaled(x, 2)
    a = v.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5
    code += 8 * torch.signbit(v).to(torch.uint8)
    code = code.reshape(x.shape)
    return code[:, 0::2] | (code[:, 1::2] << 4), s


def _blocked(s):
    """Scales (R x C) in the 128x4 blocked layout, padded with zeros."""
    R, C = s.shape
    R4, C4 = (R + 127) // 128 * 128, (C + 3) // 4 * 4
    p = torch.zeros((R4, C4), dtype=torch.uint8, device=s.device)
    p[:R, :C] = s
    return p.view(R4 // 128, 4, 32, C4 // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _unblocked(b, R, C):
    R4, C4 = (R + 127) // 128 * 128, (C + 3) // 4 * 4
    p = b[:R4 * C4].view(R4 // 128, C4 // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return p.reshape(R4, C4)[:R, :C]


def _elements(q, bits):
    if bits == 8:
        return q.view(torch.float8_e4m3fn).float()
    code = torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
    return grid[code.to(torch.int32)]


def _values(operand, bits):
    """The numbers that an operand's bytes and blocked scales stand for."""
    v = _elements(operand[0], bits)
    R, C = v.shape
    s = _unblocked(operand[1], R, C // 32).to(torch.int32)
    mult = torch.where(s == 0, 1 << 22, s << 23).view(torch.float32)
    return (v.reshape(R, C // 32, 32) * mult[..., None]).reshape(R, C)


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "cast":
        out = {}
        if "0" in case["dims"]:
            out["q0"], out["s0"] = _operand(st["x"], 4)
        if "1" in case["dims"]:
            out["q1"], out["s1"] = _operand(st["x"].t(), 4)
        return out
    if op == "dequant":
        return dict(x=_values(st["a"], 4).to(torch.bfloat16))
    if op == "product":
        c = _values(st["a"], 4) @ _values(st["b"], 4).t()
        return dict(c=c.to(torch.bfloat16 if case["out"] == "bf16" else torch.float32))
    F, a = case["F"], _values(st["a"], case["bits"])
    if op == "gated":
        g, u = (a @ _values(st[w], case["bits"]).t() for w in ("gate", "up"))
        out = dict(h=(g / (1 + torch.exp(-g)) * u).to(torch.bfloat16))
        if case["save"]:
            q, s = _operand(torch.cat([g, u], 1), 8)
            out["q"], out["s"] = q.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)
        return out
    p = a @ _values(st["b"], case["bits"]).t()
    gu = _values(st["saved"], 8) if case["saved"] == 8 else st["saved"].float()
    g, u = gu[:, :F], gu[:, F:]
    sg = 1 / (1 + torch.exp(-g))
    return dict(dgu=torch.cat([p * u * sg * (1 + g * (1 - sg)), p * g * sg], 1).to(torch.bfloat16))


# ---- the framework's entry points -------------------------------------------------

def _own(st):
    import mxfp8_block_scaled_dim0_gb300 as mx
    case = st["case"]
    op = case["op"]
    if op == "cast":
        if case["dims"] == "01":
            q0, s0, q1, s1 = mx.cast_fp4_dim0_dim1(st["x"])
            return dict(q0=q0, s0=s0, q1=q1, s1=s1)
        if case["dims"] == "0":
            q0, s0 = mx.cast_fp4_dim0(st["x"])
            return dict(q0=q0, s0=s0)
        q1, s1 = mx.cast_fp4_dim1(st["x"])
        return dict(q1=q1, s1=s1)
    if op == "dequant":
        return dict(x=mx.dequant_fp4(*st["a"]))
    if op == "product":
        return dict(c=mx.matmul_fp4(*st["a"], *st["b"],
                                    torch.bfloat16 if case["out"] == "bf16" else torch.float32))
    if op == "gated":
        w = zip(st["gate"], st["up"])
        if not case["save"]:
            return dict(h=mx.matmul_swiglu(*st["a"], *w, bits=case["bits"]))
        h, q, s = mx.matmul_swiglu(*st["a"], *w, save=True, bits=case["bits"])
        return dict(h=h, q=q.view(torch.float8_e4m3fn), s=s.view(torch.float8_e8m0fnu))
    return dict(dgu=mx.matmul_swiglu_backward(*st["a"], *st["b"], st["saved"], bits=case["bits"]))


def run(state):
    return _own(state) if own else _plain(state)


# ---- 64 bits -----------------------------------------------------------------------

def _exact_codes(x):
    """(R x C) float64 -> (e2m1 codes, exponents) of its cast along rows, from the
    definition: shared exponent floor(log2 amax) - 2, the nearest of the eight
    magnitudes, of two equally near the even one."""
    R, C = x.shape
    v = x.reshape(R, C // 32, 32)
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.where(amax == 0, -127.0, torch.frexp(amax)[1].to(torch.float64) - 3).clamp(-127, 127)
    v = v * torch.exp2(-e)
    step = torch.exp2((torch.frexp(v)[1].to(torch.float64) - 1).clamp(min=0) - 1)
    a = (torch.round(v.abs() / step) * step).clamp(max=6)
    # Codes 0..3 lie 0.5 apart, 4 and 5 one, 6 and 7 two.
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, 2 + a, 4 + a / 2)).to(torch.int32)
    return (code + 8 * torch.signbit(x).reshape(v.shape)).reshape(R, C), e[..., 0]


def _exact_operand4(x):
    code, e = _exact_codes(x)
    R, C = code.shape
    pairs = code.reshape(R, C // 2, 2)
    q = (pairs[..., 0] + 16 * pairs[..., 1]).to(torch.uint8)
    wide = (C // 32 + 3) // 4
    s = torch.zeros((R + 127) // 128 * wide * 512, dtype=torch.uint8, device=x.device)
    s[_blocked_at(R, C // 32, x.device)] = (e + 127).to(torch.uint8)
    return q, s


def _blocked_at(R, C, device):
    c = torch.arange(C, device=device)
    r = torch.arange(R, device=device)
    return ((r[:, None] // 128) * ((C + 3) // 4) + c // 4) * 512 + (r[:, None] % 32) * 16 \
        + (r[:, None] % 128) // 32 * 4 + c % 4


def _exact_values(operand, bits):
    """Bytes and blocked e8m0 scales as float64, bit field by bit field."""
    b = operand[0].to(torch.int32)
    if bits == 4:
        b = torch.stack([b % 16, b // 16], -1).reshape(b.shape[0], -1)
        ex, man, sign = (b >> 1) & 3, (b & 1).to(torch.float64) / 2, b >= 8
        mag = torch.where(ex == 0, man, (1 + man) * torch.exp2(ex.to(torch.float64) - 1))
    else:
        ex, man, sign = (b >> 3) & 15, (b & 7).to(torch.float64) / 8, b >= 128
        mag = torch.where(ex == 0, man / 64, (1 + man) * torch.exp2(ex.to(torch.float64) - 7))
    R, C = b.shape
    scale = torch.exp2(operand[1][_blocked_at(R, C // 32, b.device)].to(torch.float64) - 127)
    v = torch.where(sign, -mag, mag)
    return (v.reshape(R, C // 32, 32) * scale[..., None]).reshape(R, C)


def _exact_saved(x):
    """The e4m3 numbers of x's MX-FP8 cast along rows, scales aside."""
    R, C = x.shape
    v = x.reshape(R, C // 32, 32)
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.where(amax == 0, -127.0, torch.frexp(amax)[1].to(torch.float64) - 9).clamp(-127, 127)
    v = v * torch.exp2(-e)
    step = torch.exp2((torch.frexp(v)[1].to(torch.float64) - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448).reshape(R, C)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "cast":
        x, out = st["x"].to(torch.float64), {}
        if "0" in case["dims"]:
            out["q0"], out["s0"] = _exact_operand4(x)
        if "1" in case["dims"]:
            out["q1"], out["s1"] = _exact_operand4(x.t().contiguous())
        return out
    if op == "dequant":
        return dict(x=_exact_values(st["a"], 4))
    bits = case.get("bits", 4)
    a = _exact_values(st["a"], bits)
    if op == "gated":
        g, u = (torch.mm(a, _exact_values(st[w], bits).t()) for w in ("gate", "up"))
        out = dict(h=g * torch.sigmoid(g) * u)
        if case["save"]:
            out["q"], out["s"] = _exact_saved(torch.cat([g, u], 1)), None
        return out
    p = torch.mm(a, _exact_values(st["b"], bits).t())
    if op == "product":
        return dict(c=p)
    F = case["F"]
    gu = _exact_values(st["saved"], 8) if case["saved"] == 8 else st["saved"].to(torch.float64)
    g, u = gu.split(F, 1)
    sg = torch.sigmoid(g)
    return dict(dgu=torch.cat([p * u * (sg + g * sg * (1 - sg)), p * g * sg], 1))
