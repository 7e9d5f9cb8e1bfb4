"""Refusals of the training operators' C entry points, before any CUDA call."""
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
    def call(qa=A, sa=A, qb=A, sb=A, M=64, N=64, K=64, out=A, t=0):
        return lib.mx_matmul(qa, sa, qb, sb, M, N, K, out, t, None)
    for name in ("qa", "sa", "qb", "sb", "out"):
        assert call(**{name: None}) == mx.MX_ERR_NULL
        assert call(**{name: B}) == mx.MX_ERR_ALIGN
    for bad in (dict(M=0), dict(N=0), dict(N=-1), dict(K=0), dict(K=48), dict(K=-32),
                dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31)):
        assert call(**bad) == mx.MX_ERR_SHAPE
    assert call(t=2) == mx.MX_ERR_TYPE and call(t=-1) == mx.MX_ERR_TYPE
    assert lib.mx_strerror(mx.MX_ERR_TYPE) != lib.mx_strerror(-99)
