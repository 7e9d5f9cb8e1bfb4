"""The tests' plain 64-bit backward formulas against differences of the forward
ones (no GPU)."""
import torch

import plain64

F64 = torch.float64


def _differ(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_layer_norm_backward_formula():
    g = torch.Generator().manual_seed(3)
    M, D, eps = 5, 37, 1e-5
    x, dy, v = (torch.randn(M, D, generator=g, dtype=F64) for _ in range(3))
    w, b = (torch.randn(D, generator=g, dtype=F64) for _ in range(2))
    _, mean, rstd = plain64.layer_norm(x, w, b, eps)
    (dx, dw, db), _ = plain64.layer_norm_backward(dy, x, w, mean, rstd)
    loss = lambda x, w, b: (plain64.layer_norm(x, w, b, eps)[0] * dy).sum()  # noqa: E731
    assert abs((dx * v).sum() - _differ(lambda t: loss(t, w, b), x, v)) < 1e-7
    assert abs((dw * v[0]).sum() - _differ(lambda t: loss(x, t, b), w, v[0])) < 1e-7
    assert abs((db * v[0]).sum() - _differ(lambda t: loss(x, w, t), b, v[0])) < 1e-7


def test_swiglu_backward_formula():
    g = torch.Generator().manual_seed(4)
    gu, v = (3 * torch.randn(7, 26, generator=g, dtype=F64) for _ in range(2))
    dh = torch.randn(7, 13, generator=g, dtype=F64)
    got = (plain64.swiglu_backward(dh, gu) * v).sum()
    assert abs(got - _differ(lambda t: (plain64.swiglu(t) * dh).sum(), gu, v)) < 1e-6
