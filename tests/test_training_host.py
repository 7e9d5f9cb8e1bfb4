"""Refusals of the training operators, before any CUDA call: their C entry points
and their allocating wrappers."""
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from mxfp8_block_scaled_dim0_gb300 import build as mxbuild
import pytest

# Fake, never-dereferenced device addresses: argument checks come first.
A = 1 << 20          # 16-byte aligned
B = (1 << 20) + 8    # misaligned


@pytest.fixture(scope="module")
def lib():
    mxbuild.build()
    return mx.library()


def test_matmul_refuses(lib):
    def call(qa=A, sa=A, qb=A, sb=A, M=64, N=64, K=64, orders=0, out=A, t=0):
        return lib.mx_matmul(qa, sa, qb, sb, M, N, K, orders, out, t, None)
    for name in ("qa", "sa", "qb", "sb", "out"):
        assert call(**{name: None}) == mx.MX_ERR_NULL
        assert call(**{name: B}) == mx.MX_ERR_ALIGN
    for bad in (dict(M=0), dict(N=0), dict(N=-1), dict(K=0), dict(K=48), dict(K=-32),
                dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31)):
        assert call(**bad) == mx.MX_ERR_SHAPE
    assert call(orders=1, M=40) == mx.MX_ERR_SHAPE and call(orders=2, N=24) == mx.MX_ERR_SHAPE
    for bad in (dict(t=2), dict(t=-1), dict(orders=4), dict(orders=-1)):
        assert call(**bad) == mx.MX_ERR_TYPE
    assert lib.mx_strerror(mx.MX_ERR_TYPE) != lib.mx_strerror(-99)


def test_layer_norm_refuses(lib):
    def call(x=A, w=A, b=A, t=1, M=8, D=64, eps=1e-5, y=A, mean=A, rstd=A, q=A, s=A):
        return lib.mx_layer_norm(x, w, b, t, M, D, eps, y, mean, rstd, q, s, None)
    for name in ("x", "w", "y", "mean", "rstd", "q", "s"):
        assert call(**{name: None}) == mx.MX_ERR_NULL
    for name in ("x", "w", "b", "y", "q", "s"):
        assert call(**{name: B}) == mx.MX_ERR_ALIGN
    assert call(mean=A + 2) == mx.MX_ERR_ALIGN
    for bad in (dict(M=0), dict(D=0), dict(M=-5), dict(D=48), dict(D=16385), dict(M=1 << 31),
                dict(eps=-1.0), dict(eps=float("nan")), dict(D=16400, q=None, s=None)):
        assert call(**bad) == mx.MX_ERR_SHAPE
    assert call(t=2) == mx.MX_ERR_TYPE


def test_layer_norm_backward_refuses(lib):
    def call(dy=A, x=None, q=A, s=A, w=A, t=0, mean=A, rstd=A, M=8, D=64, dx=A, dw=A, db=A, work=A):
        return lib.mx_layer_norm_backward(dy, x, q, s, w, t, mean, rstd, M, D, dx, dw, db, work, None)
    for name in ("dy", "q", "s", "w", "mean", "rstd", "dx", "dw", "work"):
        assert call(**{name: None}) == mx.MX_ERR_NULL
    assert call(q=None, s=None) == mx.MX_ERR_NULL      # no input at all
    assert call(x=A) == mx.MX_ERR_NULL                 # two inputs
    for name in ("dy", "q", "s", "w", "dx", "dw", "db", "work"):
        assert call(**{name: B}) == mx.MX_ERR_ALIGN
    for bad in (dict(M=0), dict(D=0), dict(D=48), dict(D=16416), dict(M=1 << 31)):
        assert call(**bad) == mx.MX_ERR_SHAPE
    assert call(t=7) == mx.MX_ERR_TYPE
    assert mx.mx_layer_norm_backward_work_bytes(1, 8) == 64
    assert mx.mx_layer_norm_backward_work_bytes(-1, 8) == -1


def test_swiglu_refuses(lib):
    def fwd(gu=A, M=8, F=64, h=A, q=A, s=A):
        return lib.mx_swiglu(gu, M, F, h, q, s, None)

    def back(dh=A, gu=None, q=A, s=A, M=8, F=64, out=A):
        return lib.mx_swiglu_backward(dh, gu, q, s, M, F, out, None)
    for name in ("gu", "h", "q", "s"):
        assert fwd(**{name: None}) == mx.MX_ERR_NULL and fwd(**{name: B}) == mx.MX_ERR_ALIGN
    for name in ("dh", "q", "s", "out"):
        assert back(**{name: None}) == mx.MX_ERR_NULL and back(**{name: B}) == mx.MX_ERR_ALIGN
    assert back(gu=A) == mx.MX_ERR_NULL and back(q=None, s=None) == mx.MX_ERR_NULL
    for bad in (dict(M=0), dict(F=0), dict(F=48), dict(M=1 << 31), dict(F=(1 << 24) + 32)):
        assert fwd(**bad) == mx.MX_ERR_SHAPE and back(**bad) == mx.MX_ERR_SHAPE


def test_wrappers_refuse_cpu_tensors_and_wrong_types(lib):
    x, w = torch.zeros(64, 96, dtype=torch.bfloat16), torch.zeros(96)
    q, s = torch.zeros(64, 96, dtype=torch.uint8), torch.zeros(128 * 4, dtype=torch.uint8)
    stats = torch.zeros(64)
    for call in (lambda: mx.layer_norm(x, w), lambda: mx.layer_norm(x, w, save=True),
                 lambda: mx.layer_norm_backward(x, x, w, stats, stats),
                 lambda: mx.layer_norm_backward(x, (q, s), w, stats, stats),
                 lambda: mx.swiglu(x), lambda: mx.swiglu(x, save=False),
                 lambda: mx.swiglu_backward(x[:, :48].contiguous(), x),
                 lambda: mx.matmul(q, s, q, s), lambda: mx.cast_dim0(x), lambda: mx.cast_dim1(x),
                 lambda: mx.cast_dim0_dim1(x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: mx.layer_norm(x.float(), w), lambda: mx.layer_norm(x, w.double()),
                 lambda: mx.layer_norm(x, w, w.to(torch.bfloat16)),
                 lambda: mx.swiglu(x.half()), lambda: mx.swiglu_backward(x.float(), x),
                 lambda: mx.matmul(x, s, q, s), lambda: mx.matmul(q, s, q, s, torch.float16)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: mx.layer_norm(x.t(), w), lambda: mx.layer_norm(x, w[:5]),
                 lambda: mx.layer_norm_backward(x, x, w, stats[:3], stats),
                 lambda: mx.layer_norm_backward(x, (q[:5], s), w, stats, stats),
                 lambda: mx.swiglu(x[:, :33].contiguous()), lambda: mx.swiglu_backward(x, x),
                 lambda: mx.matmul(q, s, q[:, :64].contiguous(), s),
                 lambda: mx.matmul(q, s[:9], q, s)):
        with pytest.raises(ValueError):
            call()
