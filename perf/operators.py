"""Measured cases of the operators that train a layer from 8-bit saved
activations: layer norm and gated SiLU, forward and backward, with their
inputs saved as MX-FP8, and the MX product that linear layers use on such
operands.

``own`` false: every operator in plain form, elementary torch operations in 32
bits, rounded once at the end.  ``own`` true: the framework's entry points.
``exact`` computes the same results in 64 bits, from the definitions.
"""
import math

import torch

own = False

EPS = 1e-5
DEV = "cuda"


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # One token through a norm while decoding: launch latency.
        dict(name="norm 1x4096", op="norm", M=1, D=4096, save=False, wtype="bf16"),
        # The norm ahead of the MoE activations' layer, its input saved in 8 bits.
        dict(name="norm save 16640x5120", op="norm", M=16640, D=5120, save=True, wtype="f32"),
        # Its backward pass from the 8-bit saved input.
        dict(name="norm back 8-bit 16640x5120", op="norm_back", M=16640, D=5120, save=True,
             wtype="f32"),
        # Backward from a bf16 input, a micro-batch of 4096 tokens.
        dict(name="norm back 4096x4096", op="norm_back", M=4096, D=4096, save=False, wtype="bf16"),
        # Odd sizes: a head-less width and a ragged batch.
        dict(name="norm back 1031x1021", op="norm_back", M=1031, D=1021, save=False, wtype="f32"),
        # Gated activation of one packed sequence, input saved in 8 bits.
        dict(name="swiglu save 1024x4096", op="swiglu", M=1024, F=4096, save=True),
        # The expert layer's width at the MoE token count.
        dict(name="swiglu save 16640x8192", op="swiglu", M=16640, F=8192, save=True),
        # Backward of the same from the saved bytes.
        dict(name="swiglu back 8-bit 16640x8192", op="swiglu_back", M=16640, F=8192, save=True),
        # Backward from bf16 with a width that no vector divides.
        dict(name="swiglu back 515x2731", op="swiglu_back", M=515, F=2731, save=False),
        # Forward product of a small layer on a few tokens: latency.
        dict(name="product 160x1024x1024", op="product", M=160, N=1024, K=1024, out="bf16"),
        # Forward product of the expert weights (8192 x 5120) on all tokens.
        dict(name="product 16640x8192x5120", op="product", M=16640, N=8192, K=5120, out="bf16"),
        # Weight gradient of that layer from its 8-bit saved input: the
        # gradient is cast along the tokens, then multiplied.
        dict(name="wgrad 16640x8192x5120", op="wgrad", M=16640, N=8192, K=5120, out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "swiglu", "swiglu_back", "product", "wgrad"])
    save = rng.random() < 0.5
    if op in ("norm", "norm_back"):
        D = _log(rng, 32, 16384)
        M = min(_log(rng, 1, 16640), 16640 * 5120 // D)
        if save:
            D = max(32, D // 32 * 32)
        elif rng.random() < 0.5:
            D = max(32, D // 8 * 8)
        return dict(op=op, M=M, D=D, save=save, wtype=rng.choice(["bf16", "f32"]))
    if op in ("swiglu", "swiglu_back"):
        F = _log(rng, 32, 16384)
        M = min(_log(rng, 1, 16640), 16640 * 8192 // F)
        if save:
            F = max(32, F // 32 * 32)
        elif rng.random() < 0.5:
            F = max(32, F // 8 * 8)
        return dict(op=op, M=M, F=F, save=save)
    M = _log(rng, 1, 16640)
    N = _log(rng, 32, 8192)
    K = max(32, _log(rng, 32, 8192) // 32 * 32)
    if op == "wgrad":
        M, N = max(32, M // 32 * 32), max(32, N // 32 * 32)
    return dict(op=op, M=M, N=N, K=min(K, 5120), out=rng.choice(["bf16", "f32"]))


def work(case):
    op, M = case["op"], case["M"]
    if op in ("norm", "norm_back"):
        D = case["D"]
        w = (4 if case["wtype"] == "f32" else 2) * D
        saved = M * D + M * D / 32
        if op == "norm":
            return {"bytes": 4 * M * D + 8 * M + 2 * w + (saved if case["save"] else 0),
                    "flops": 10 * M * D}
        x = saved if case["save"] else 2 * M * D
        return {"bytes": 4 * M * D + x + 8 * M + 3 * w, "flops": 16 * M * D}
    if op in ("swiglu", "swiglu_back"):
        F = case["F"]
        saved = 2 * M * F + 2 * M * F / 32
        if op == "swiglu":
            return {"bytes": 6 * M * F + (saved if case["save"] else 0), "flops": 8 * M * F}
        return {"bytes": 6 * M * F + (saved if case["save"] else 4 * M * F), "flops": 14 * M * F}
    N, K = case["N"], case["K"]
    size = 2 if case["out"] == "bf16" else 4
    if op == "product":
        return {"bytes": (M + N) * K * 33 / 32 + size * M * N, "flops": 2 * M * N * K}
    return {"bytes": 2 * M * N + M * K * 33 / 32 + size * N * K, "flops": 2 * M * N * K}


# ---- inputs --------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _hidden(g, M, D):
    """A residual stream: a small mean, some loud channels, tokens of uneven size."""
    x = _randn(g, M, D).mul_(torch.exp(0.5 * _randn(g, 1, D))).add_(0.1)
    return x.mul_(torch.exp(0.3 * _randn(g, M, 1))).to(torch.bfloat16)


def _gradient(g, M, D):
    return _randn(g, M, D).mul_(1e-3 * torch.exp(0.5 * _randn(g, M, 1))).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, M = case["op"], case["M"]
    st = dict(case=case)
    if op in ("norm", "norm_back"):
        D = case["D"]
        wt = torch.float32 if case["wtype"] == "f32" else torch.bfloat16
        x = _hidden(g, M, D)
        st["w"] = (1 + 0.1 * _randn(g, D)).to(wt)
        st["b"] = (0.1 * _randn(g, D)).to(wt)
        if op == "norm":
            st["x"] = x
        else:
            st["dy"] = _gradient(g, M, D)
            xf = x.float()
            st["mean"] = xf.mean(-1)
            st["rstd"] = torch.rsqrt((xf - st["mean"][:, None]).square().mean(-1) + EPS)
            if case["save"]:
                q, s = _cast_rows(x)
                st["q"], st["s"] = q.view(torch.uint8), _blocked(s)
            else:
                st["x"] = x
    elif op in ("swiglu", "swiglu_back"):
        F = case["F"]
        gu = (1.5 * _randn(g, M, 2 * F)).to(torch.bfloat16)
        if op == "swiglu_back":
            st["dh"] = _gradient(g, M, F)
        if op == "swiglu_back" and case["save"]:
            q, s = _cast_rows(gu)
            st["q"], st["s"] = q.view(torch.uint8), _blocked(s)
        else:
            st["gu"] = gu
    elif op == "product":
        for name, rows, x in (("a", M, _hidden(g, M, case["K"])),
                              ("b", case["N"], (0.02 * _randn(g, case["N"], case["K"])).to(torch.bfloat16))):
            q, s = _cast_rows(x)
            st["q" + name], st["s" + name] = q.view(torch.uint8), _blocked(s)
    else:
        st["dy"] = _gradient(g, M, case["N"])
        q, s = _cast_rows(_hidden(g, M, case["K"]).t())
        st["q"], st["s"] = q.view(torch.uint8), _blocked(s)
    return st


# ---- plain forms ---------------------------------------------------------------

def _cast_rows(x):
    """MX cast of x (R x C) along its rows: e4m3 values (R x C) and scale
    bytes (R x C/32)."""
    R, C = x.shape
    v = x.float().reshape(R, C // 32, 32)
    e = v.abs().amax(-1).view(torch.int32) >> 23
    s = (e - 8).clamp(min=0)
    mult = ((254 - s) << 23).view(torch.float32)
    q = (v * mult[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.reshape(R, C), s.to(torch.uint8)


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


def _values(q, s_blk):
    """The numbers that e4m3 bytes (R x C) and their blocked scales stand for."""
    R, C = q.shape
    s = _unblocked(s_blk, R, C // 32).to(torch.int32)
    mult = torch.where(s == 0, 1 << 22, s << 23).view(torch.float32)
    v = q.view(torch.float8_e4m3fn).float().reshape(R, C // 32, 32)
    return (v * mult[..., None]).reshape(R, C)


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "norm":
        x = st["x"].float()
        mean = x.mean(-1)
        d = x - mean[:, None]
        rstd = torch.rsqrt(d.square().mean(-1) + EPS)
        y = (d * rstd[:, None] * st["w"].float() + st["b"].float()).to(torch.bfloat16)
        out = dict(y=y, mean=mean, rstd=rstd)
        if case["save"]:
            out["q"], s = _cast_rows(st["x"])
            out["s"] = _blocked(s)
        return out
    if op == "norm_back":
        x = _values(st["q"], st["s"]) if case["save"] else st["x"].float()
        dy = st["dy"].float()
        xh = (x - st["mean"][:, None]) * st["rstd"][:, None]
        gr = dy * st["w"].float()
        dx = gr - gr.mean(-1)[:, None] - xh * (gr * xh).mean(-1)[:, None]
        dx = (st["rstd"][:, None] * dx).to(torch.bfloat16)
        wt = st["w"].dtype
        return dict(dx=dx, dw=(dy * xh).sum(0).to(wt), db=dy.sum(0).to(wt))
    if op == "swiglu":
        F = case["F"]
        gu = st["gu"].float()
        g, u = gu[:, :F], gu[:, F:]
        out = dict(h=(g / (1 + torch.exp(-g)) * u).to(torch.bfloat16))
        if case["save"]:
            out["q"], s = _cast_rows(st["gu"])
            out["s"] = _blocked(s)
        return out
    if op == "swiglu_back":
        F = case["F"]
        gu = _values(st["q"], st["s"]) if case["save"] else st["gu"].float()
        g, u = gu[:, :F], gu[:, F:]
        dh = st["dh"].float()
        sg = 1 / (1 + torch.exp(-g))
        dg = dh * u * sg * (1 + g * (1 - sg))
        du = dh * g * sg
        return dict(dgu=torch.cat([dg, du], 1).to(torch.bfloat16))
    ot = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    if op == "product":
        a, b = _values(st["qa"], st["sa"]), _values(st["qb"], st["sb"])
        return dict(c=(a @ b.t()).to(ot))
    q, s = _cast_rows(st["dy"].t())
    dy = _values(q.view(torch.uint8), _blocked(s))
    return dict(dw=(dy @ _values(st["q"], st["s"]).t()).to(ot))


# ---- the framework's entry points -------------------------------------------------

def _own(st):
    import mxfp8_block_scaled_dim0_gb300 as mx
    case = st["case"]
    op = case["op"]
    if op == "norm":
        if not case["save"]:
            y, mean, rstd = mx.layer_norm(st["x"], st["w"], st["b"], EPS)
            return dict(y=y, mean=mean, rstd=rstd)
        y, mean, rstd, q, s = mx.layer_norm(st["x"], st["w"], st["b"], EPS, save=True)
        return dict(y=y, mean=mean, rstd=rstd, q=q.view(torch.float8_e4m3fn), s=s)
    if op == "norm_back":
        saved = (st["q"], st["s"]) if case["save"] else st["x"]
        dx, dw, db = mx.layer_norm_backward(st["dy"], saved, st["w"], st["mean"], st["rstd"])
        return dict(dx=dx, dw=dw, db=db)
    if op == "swiglu":
        if not case["save"]:
            return dict(h=mx.swiglu(st["gu"]))
        h, q, s = mx.swiglu(st["gu"], save=True)
        return dict(h=h, q=q.view(torch.float8_e4m3fn), s=s)
    if op == "swiglu_back":
        saved = (st["q"], st["s"]) if case["save"] else st["gu"]
        return dict(dgu=mx.swiglu_backward(st["dh"], saved))
    ot = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    if op == "product":
        return dict(c=mx.matmul(st["qa"], st["sa"], st["qb"], st["sb"], ot))
    q, s = mx.cast_dim1(st["dy"])
    return dict(dw=mx.matmul(q, s, st["q"], st["s"], ot))


def run(state):
    return _own(state) if own else _plain(state)


# ---- 64 bits -----------------------------------------------------------------------

def _exact_cast(x):
    """(R x C) float64 -> what its MX cast along rows stands for, from the
    definition: shared exponent floor(log2 amax) - 8, elements on the e4m3
    grid (spacing 2^(max(floor(log2 |v|), -6) - 3), ties to even, +-448)."""
    R, C = x.shape
    v = x.reshape(R, C // 32, 32)
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.frexp(amax)[1].to(torch.float64) - 9
    e = torch.where(amax == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    v = v * torch.exp2(-e)
    step = torch.exp2((torch.frexp(v)[1].to(torch.float64) - 1).clamp(min=-6) - 3)
    v = (torch.round(v / step) * step).clamp(-448, 448)
    return v, e


def _exact_values(q, s_blk):
    """e4m3 bytes and blocked e8m0 scales as float64, bit field by bit field."""
    R, C = q.shape
    c = torch.arange(C // 32, device=q.device)
    r = torch.arange(R, device=q.device)
    wide = (C // 32 + 3) // 4
    at = ((r[:, None] // 128) * wide + c // 4) * 512 + (r[:, None] % 32) * 16 \
        + (r[:, None] % 128) // 32 * 4 + c % 4
    scale = torch.exp2(s_blk[at].to(torch.float64) - 127)
    b = q.to(torch.int32)
    ex, man = (b >> 3) & 15, (b & 7).to(torch.float64)
    mag = torch.where(ex == 0, man / 512,
                      (1 + man / 8) * torch.exp2(ex.to(torch.float64) - 7))
    v = torch.where(b >= 128, -mag, mag)
    return (v.reshape(R, C // 32, 32) * scale[..., None]).reshape(R, C)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "norm":
        x = st["x"].to(f64)
        D = x.shape[1]
        mean = x.sum(-1) / D
        var = ((x - mean[:, None]) ** 2).sum(-1) / D
        rstd = (var + EPS) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None] * st["w"].to(f64) + st["b"].to(f64)
        out = dict(y=y, mean=mean, rstd=rstd)
        if case["save"]:
            out["q"], out["s"] = _exact_cast(x)[0].reshape(x.shape), None
        return out
    if op == "norm_back":
        x = _exact_values(st["q"], st["s"]) if case["save"] else st["x"].to(f64)
        dy, w = st["dy"].to(f64), st["w"].to(f64)
        D = x.shape[1]
        rstd = st["rstd"].to(f64)[:, None]
        xh = (x - st["mean"].to(f64)[:, None]) * rstd
        c1 = (dy @ w / D)[:, None]
        c2 = ((dy * xh) @ w / D)[:, None]
        return dict(dx=rstd * (dy * w - c1 - xh * c2), dw=(dy * xh).sum(0), db=dy.sum(0))
    if op in ("swiglu", "swiglu_back"):
        F = case["F"]
        gu = _exact_values(st["q"], st["s"]) if "q" in st else st["gu"].to(f64)
        g, u = gu.split(F, 1)
        sg = torch.sigmoid(g)
        if op == "swiglu":
            out = dict(h=g * sg * u)
            if case["save"]:
                out["q"], out["s"] = _exact_cast(gu)[0].reshape(gu.shape), None
            return out
        dh = st["dh"].to(f64)
        return dict(dgu=torch.cat([dh * u * (sg + g * sg * (1 - sg)), dh * g * sg], 1))
    if op == "product":
        a, b = _exact_values(st["qa"], st["sa"]), _exact_values(st["qb"], st["sb"])
        return dict(c=torch.mm(a, b.t()))
    v, e = _exact_cast(st["dy"].t().to(f64))
    dy = (v * torch.exp2(e)).reshape(case["N"], case["M"])
    return dict(dw=torch.mm(dy, _exact_values(st["q"], st["s"]).t()))
