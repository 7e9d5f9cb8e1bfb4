"""The plain 64-bit forms of plain_fp4.py on the CPU: MX-FP4 against hand-worked blocks and
brute force, the gradient of the joined products against differences and against autograd."""
import torch

from plain64 import F64
from plain_fp4 import GRID, cast_rows, codes_of, e2m1_values, mx4_values, swiglu_back_of, swiglu_of


def block(*head):
    x = torch.zeros(1, 32, dtype=torch.bfloat16)
    x[0, :len(head)] = torch.tensor(head, dtype=torch.bfloat16)
    return x


def cast(x):
    q, s = cast_rows(x)
    return codes_of(q)[0].tolist(), int(s[0])


def test_hand_worked_blocks():
    # amax 6 = 1.5 2^2: scale 2^0; every magnitude, both signs.
    codes, s = cast(block(6, 4, 3, 2, 1.5, 1, 0.5, -0.5, -6, -0.0))
    assert s == 127 and codes[:10] == [7, 6, 5, 4, 3, 2, 1, 9, 15, 8] and not any(codes[10:])
    # Ties go to the even code: 5 -> 4, 3.5 -> 4, 2.5 -> 2, 1.75 -> 2, 1.25 -> 1, 0.75 -> 1, 0.25 -> 0.
    assert cast(block(4, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25))[0][:8] == [6, 6, 6, 4, 4, 2, 2, 0]
    # 7.5 stays with 4's scale and saturates; 8 takes the next.
    assert cast(block(7.5, 1)) == ([7, 2] + [0] * 30, 127)
    assert cast(block(8, 1)) == ([6, 1] + [0] * 30, 128)
    # The smallest scale is 2^-127, and holds subnormals.
    assert cast(block(2.0 ** -126, 2.0 ** -127, 2.0 ** -128))[1] == 0
    assert cast(block(2.0 ** -126, 2.0 ** -127, 2.0 ** -128))[0][:3] == [4, 2, 1]
    assert cast(block()) == ([0] * 32, 0)
    for bad in (float("inf"), float("nan"), -float("inf")):
        assert cast(block(1, bad)) == ([7] * 32, 255)


def test_casts_are_nearest():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(64, 96, generator=g) * torch.exp2(torch.randint(-30, 30, (64, 1), generator=g).float())
         ).to(torch.bfloat16)
    q, s = cast_rows(x)
    v = mx4_values(q, s)
    scale = torch.exp2(torch.frexp(x.to(F64).reshape(64, 3, 32).abs().amax(-1))[1].to(F64) - 3)[..., None]
    grid = torch.tensor([-a for a in GRID[:0:-1]] + list(GRID), dtype=F64)
    near = (x.to(F64).reshape(64, 3, 32, 1) / scale[..., None] - grid).abs().amin(-1)
    assert torch.equal(((x.to(F64) - v).reshape(64, 3, 32) / scale).abs(), near)


def test_packed_codes():
    q = torch.arange(256, dtype=torch.uint8)[None]
    v = e2m1_values(q)[0]
    for b in range(256):
        for k, code in enumerate((b & 15, b >> 4)):
            want = GRID[code & 7] * (-1 if code & 8 else 1)
            assert float(v[2 * b + k]) == want


def test_gradient_against_differences():
    g = torch.Generator().manual_seed(2)
    M, D, F = 3, 5, 4
    gu = (2 * torch.randn(M, 2 * F, generator=g, dtype=F64))
    w2, dy = torch.randn(D, F, generator=g, dtype=F64), torch.randn(M, D, generator=g, dtype=F64)
    none = torch.zeros(M, 2 * F, dtype=F64)

    def loss(p):
        return float(((swiglu_of(p, none)[0] @ w2.t()) * dy).sum())
    dh = dy @ w2
    dgu = swiglu_back_of(dh, torch.zeros_like(dh), gu)[0]
    for i in range(M):
        for j in range(2 * F):
            up, down = gu.clone(), gu.clone()
            up[i, j] += 1e-5
            down[i, j] -= 1e-5
            # central differences: h^2 / 6 of the third derivative, and rounding 1e-16 / h
            assert abs((loss(up) - loss(down)) / 2e-5 - float(dgu[i, j])) < 1e-8
    leaf = gu.clone().requires_grad_()
    a, b = leaf.chunk(2, -1)
    ((a * torch.sigmoid(a) * b) @ w2.t() * dy).sum().backward()
    assert float((leaf.grad - dgu).abs().max()) < 1e-12


def test_tolerances_hold_what_they_promise():
    """Sums moved by up to their tolerance move the results by no more than theirs."""
    g = torch.Generator().manual_seed(3)
    p = 3 * torch.randn(200, 64, generator=g, dtype=F64)
    for size in (1e-6, 1e-2):
        tol = size * p.abs() + size / 10
        h, room = swiglu_of(p, tol)
        for _ in range(5):
            moved = p + tol * (2 * torch.rand(p.shape, generator=g, dtype=F64) - 1)
            assert bool(((swiglu_of(moved, tol)[0] - h).abs() <= room).all())
    dh = torch.randn(200, 32, generator=g, dtype=F64)
    tol = 1e-3 * dh.abs()
    want, room = swiglu_back_of(dh, tol, p)
    moved = swiglu_back_of(dh + tol * (2 * torch.rand(dh.shape, generator=g, dtype=F64) - 1), tol, p)[0]
    assert bool(((moved - want).abs() <= room).all())
