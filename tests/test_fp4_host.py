"""Refusals of the 4-bit and gated entry points, before any CUDA call, and of their
wrappers."""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from mxfp8_block_scaled_dim0_gb300 import build as mxbuild

A = 1 << 20          # fake, never-dereferenced device addresses: 16-byte aligned
B = (1 << 20) + 8    # misaligned
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    mxbuild.build()
    return mx.library()


def refuses(call, null, aligned, shapes, types=()):
    for name in null:
        assert call(**{name: None}) == mx.MX_ERR_NULL, name
    for name in aligned:
        assert call(**{name: B}) == mx.MX_ERR_ALIGN, name
    for bad in shapes:
        assert call(**bad) == mx.MX_ERR_SHAPE, bad
    for bad in types:
        assert call(**bad) == mx.MX_ERR_TYPE, bad


def test_casts_refuse(lib):
    def one(fn):
        return lambda x=A, M=64, K=64, q=A, s=A: fn(x, M, K, q, s, None)
    sizes = [dict(K=0), dict(K=48), dict(K=-32), dict(M=0), dict(M=-1), dict(M=BIG), dict(K=BIG)]
    refuses(one(lib.mx_cast_fp4_dim0), "xqs", "xqs", sizes)
    refuses(one(lib.mx_cast_fp4_dim1), "xqs", "xqs", sizes + [dict(M=33)])

    def both(x=A, M=64, K=64, q0=A, s0=A, q1=A, s1=A):
        return lib.mx_cast_fp4_dim0_dim1(x, M, K, q0, s0, q1, s1, None)
    names = ("x", "q0", "s0", "q1", "s1")
    refuses(both, names, names, sizes + [dict(M=33)])

    def back(q=A, R=3, C=64, s=A, out=A):
        return lib.mx_dequant_fp4(q, R, C, s, out, None)
    names = ("q", "s", "out")
    refuses(back, names, names, [dict(R=0), dict(C=0), dict(C=48), dict(R=BIG), dict(C=BIG)])


def test_products_refuse(lib):
    def mm(qa=A, sa=A, qb=A, sb=A, M=64, N=64, K=64, out=A, t=0):
        return lib.mx_matmul_fp4(qa, sa, qb, sb, M, N, K, out, t, None)
    names = ("qa", "sa", "qb", "sb", "out")
    refuses(mm, names, names,
            [dict(M=0), dict(N=0), dict(K=0), dict(K=32), dict(K=96), dict(M=BIG), dict(N=BIG), dict(K=BIG)],
            [dict(t=2), dict(t=-1)])

    def fwd(qx=A, sx=A, qg=A, sg=A, qu=A, su=A, M=64, F=64, K=64, f=0, h=A, q=A, s=A):
        return lib.mx_matmul_swiglu(qx, sx, qg, sg, qu, su, M, F, K, f, h, q, s, None)

    def bwd(qdy=A, sdy=A, qw=A, sw=A, M=64, F=64, K=64, f=0, gu=None, q=A, s=A, out=A):
        return lib.mx_matmul_swiglu_backward(qdy, sdy, qw, sw, M, F, K, f, gu, q, s, out, None)
    sizes = [dict(M=0), dict(F=0), dict(F=48), dict(F=16), dict(K=0), dict(K=48), dict(f=1, K=96),
             dict(f=1, K=32), dict(M=BIG), dict(K=BIG), dict(F=(1 << 24) + 32)]
    types = [dict(f=2), dict(f=-1)]
    names = ("qx", "sx", "qg", "sg", "qu", "su", "h", "q", "s")
    refuses(fwd, names, names, sizes, types)
    names = ("qdy", "sdy", "qw", "sw", "q", "s", "out")
    refuses(bwd, names, names, sizes, types)
    assert bwd(gu=A) == mx.MX_ERR_NULL                     # two inputs
    assert bwd(q=None, s=None) == mx.MX_ERR_NULL           # none
    assert bwd(gu=B, q=None, s=None) == mx.MX_ERR_ALIGN


def test_wrappers_refuse(lib):
    x = torch.zeros(64, 128, dtype=torch.bfloat16)
    q8, q4, s = (torch.zeros(n, dtype=torch.uint8) for n in ((64, 128), (64, 64), (512,)))
    w8, w4, ws = (torch.zeros(n, dtype=torch.uint8) for n in ((256, 128), (256, 64), (1024,)))
    gu = torch.zeros(64, 128, dtype=torch.bfloat16)
    on_cpu = [lambda: mx.cast_fp4_dim0(x), lambda: mx.cast_fp4_dim1(x), lambda: mx.cast_fp4_dim0_dim1(x),
              lambda: mx.dequant_fp4(q4, s), lambda: mx.matmul_fp4(q4, s, q4, s),
              lambda: mx.matmul_swiglu(q8, s, w8, ws), lambda: mx.matmul_swiglu(q4, s, w4, ws, True, 4),
              lambda: mx.matmul_swiglu(q8, s, (q8, q8), (s, s)),
              lambda: mx.matmul_swiglu_backward(q8, s, q8, s, gu.repeat(1, 1)),
              lambda: mx.matmul_swiglu_backward(q4, s, q4, s, (q8, s), 4)]
    for call in on_cpu:
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: mx.cast_fp4_dim0(x.float()), lambda: mx.dequant_fp4(x, s),
                 lambda: mx.matmul_fp4(x, s, q4, s), lambda: mx.matmul_fp4(q4, s, q4, s, torch.float16),
                 lambda: mx.matmul_fp4(q4.view(torch.float8_e4m3fn), s, q4, s),
                 lambda: mx.matmul_swiglu(x, s, w8, ws), lambda: mx.matmul_swiglu(q8, s, (q8, x), (s, s)),
                 lambda: mx.matmul_swiglu_backward(q8, s, q8, s, gu.float())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: mx.cast_fp4_dim0(x.t()), lambda: mx.dequant_fp4(q4.t(), s),
                 lambda: mx.dequant_fp4(q4, s[:9]), lambda: mx.matmul_fp4(q4, s, q4[:, :32].contiguous(), s),
                 lambda: mx.matmul_fp4(q4, s[:9], q4, s), lambda: mx.matmul_swiglu(q8, s, q8, s),
                 lambda: mx.matmul_swiglu(q8, s, w4, ws), lambda: mx.matmul_swiglu(q8, s, w8, ws, bits=6),
                 lambda: mx.matmul_swiglu(q8, s, (q8, q8[:60]), (s, s)),
                 lambda: mx.matmul_swiglu(q8, s, (q8, q4), (s, s)), lambda: mx.matmul_swiglu(q8, s, w8, ws[:600]),
                 lambda: mx.matmul_swiglu_backward(q8, s, q8, s, gu[:5]),
                 lambda: mx.matmul_swiglu_backward(q8, s, q8, s, gu, bits=16),
                 lambda: mx.mx_matmul_swiglu_backward(q8, s, q8, s, None, None, None, gu)):
        with pytest.raises(ValueError):
            call()
