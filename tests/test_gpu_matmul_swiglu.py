"""The products joined with the gated SiLU on the GPU, forward and backward, against 64
bits.  Tolerances: plain_fp4.product's for the sums, carried through the formulas by
plain_fp4.swiglu_of and swiglu_back_of."""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from plain64 import blocked_at, e4m3_values, mx_values, scale_values
from plain_fp4 import product, swiglu_back_of, swiglu_of

pytestmark = pytest.mark.gpu

GUARD = 4096
BITS = [8, 4]


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()
    assert mx.mx_watchdog(clear=True) == 0
    yield
    torch.cuda.synchronize()
    assert mx.mx_watchdog(clear=True) == 0


def operand(R, K, bits, seed, size=1.0):
    """An MX operand of normal values; the scale buffer's padding holds 0xFF, which no
    result may depend on."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (size * torch.randn(R, K, generator=g, device="cuda")
         * torch.exp(0.5 * torch.randn(R, 1, generator=g, device="cuda"))).to(torch.bfloat16)
    q, s = mx.cast_dim0(x) if bits == 8 else mx.cast_fp4_dim0(x)
    padded = torch.full_like(s, 255)
    at = blocked_at(R, K // 32, "cuda")
    padded[at] = s[at]
    return q, padded


class Guarded:
    def __init__(self, shape, dtype):
        n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
        self.all = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.mid = self.all[GUARD:GUARD + n].view(dtype).view(shape)
        self.n = n

    def check(self):
        assert bool((self.all[:GUARD] == 0xA5).all()), "written before the start"
        assert bool((self.all[GUARD + self.n:] == 0xA5).all()), "written past the end"


def off(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), "%d of %d values off" % (int(bad.sum()), bad.numel())


def check_saved(q, s_blk, p, tol):
    """Saved bytes and scales of sums p that are off by at most tol."""
    M, F2 = p.shape
    at = blocked_at(M, F2 // 32, "cuda")
    s = s_blk[at]
    pad = torch.ones_like(s_blk, dtype=torch.bool)
    pad[at] = False
    assert bool((s_blk[pad] == 0).all()), "padding scales"
    b, t = p.reshape(M, -1, 32), tol.reshape(M, -1, 32)
    hi, lo = (b.abs() + t).amax(-1), (b.abs() - t).amax(-1).clamp(min=0)
    exponent = lambda a: (torch.frexp(a)[1] - 1 - 8 + 127).clamp(0, 254)  # noqa: E731
    assert bool((s <= exponent(hi)).all()) and bool((s >= exponent(lo)).all()), "scales"
    scale = scale_values(s)[..., None]
    got = e4m3_values(q).reshape(M, -1, 32)
    want = (b / scale).clamp(-448, 448)
    half = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, device="cuda", dtype=p.dtype))
    bad = ~((got - want).abs() <= (t / scale) * (1 + 2.0 ** -4) + half)
    assert not bool(bad.any()), "%d saved values off" % int(bad.sum())


def forward(M, F, K, bits, save, seed=0, size=None):
    """Returns the operands (x, gate, up) and h."""
    x = operand(M, K, bits, seed + M + K)
    gate, up = (operand(F, K, bits, seed + F + i, (size or 1.5) * K ** -0.5) for i in range(2))
    h = Guarded((M, F), torch.bfloat16)
    pg, pu = product(x, gate, bits), product(x, up, bits)
    p, tol = torch.cat([pg[0], pu[0]], 1), torch.cat([pg[2], pu[2]], 1)
    if save:
        q = Guarded((M, 2 * F), torch.uint8)
        s = Guarded((mx.mx_blocked_bytes(M, 2 * F // 32),), torch.uint8)
        mx.mx_matmul_swiglu(*x, *gate, *up, h.mid, q.mid, s.mid, bits=bits)
        torch.cuda.synchronize()
        q.check()
        s.check()
        check_saved(q.mid, s.mid, p, tol)
    else:
        mx.mx_matmul_swiglu(*x, *gate, *up, h.mid, bits=bits)
        torch.cuda.synchronize()
    h.check()
    off(h.mid, *swiglu_of(p, tol))
    return x, gate, up, h.mid


@pytest.mark.parametrize("save", [False, True], ids=["plain", "save"])
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,F,K", [
    (128, 128, 256), (1, 128, 64), (1, 1024, 2048), (3, 256, 576), (130, 384, 192), (515, 1024, 320),
    (33, 8192, 128), (700, 128, 4160)])
def test_forward(M, F, K, bits, save):
    forward(M, F, K, bits, save)


@pytest.mark.parametrize("save", [False, True], ids=["plain", "save"])
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,F,K", [(256, 4096, 256), (2050, 1024, 448), (1031, 2048, 64), (2304, 2304, 1088)])
def test_forward_in_pairs(M, F, K, bits, save):
    forward(M, F, K, bits, save)


@pytest.mark.parametrize("save", [False, True], ids=["plain", "save"])
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,F,K", [(1, 64, 64), (20, 192, 320), (5, 32, 64), (200, 96, 576), (130, 160, 1088),
                                   (2, 2720, 1024), (515, 2720, 256), (1031, 2784, 448), (2060, 4000, 192),
                                   (2304, 2208, 128)])
def test_widths_off_the_scale_tile(M, F, K, bits, save):
    """The last scale tile, box and saved scales of a row are partial."""
    forward(M, F, K, bits, save)


@pytest.mark.parametrize("K", [32, 96, 160, 1056])
@pytest.mark.parametrize("M,F", [(5, 160), (1031, 2816)])
def test_forward_of_8_bits_with_odd_blocks(M, F, K):
    forward(M, F, K, 8, True)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,F,K", [(70, 96, 16640), (1, 64, 65536), (200, 128, 8256), (1200, 2080, 8256),
                                   (2304, 2304, 16640)])
def test_long_sums_saved(M, F, K, bits):
    """Contractions in several runs."""
    forward(M, F, K, bits, True)
    forward(M, F, K, bits, False)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,F", [(40, 256), (2304, 2304)])
def test_steep_gates(M, F, bits):
    """Gates far beyond where the sigmoid leaves fp32's normal range."""
    forward(M, F, 256, bits, True, size=60.0)


def backward(M, F, K, bits, saved, seed=0, size=1.5):
    dy = operand(M, K, bits, seed + M + K, 1e-3)
    w = operand(F, K, bits, seed + F, K ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    gu = (size * torch.randn(M, 2 * F, generator=g, device="cuda")).to(torch.bfloat16)
    out = Guarded((M, 2 * F), torch.bfloat16)
    if saved == 8:
        q, s = mx.cast_dim0(gu)
        padded = torch.full_like(s, 255)
        at = blocked_at(M, 2 * F // 32, "cuda")
        padded[at] = s[at]
        mx.mx_matmul_swiglu_backward(*dy, *w, None, q, padded, out.mid, bits=bits)
        gu = mx_values(q, padded)
    else:
        mx.mx_matmul_swiglu_backward(*dy, *w, gu, None, None, out.mid, bits=bits)
    torch.cuda.synchronize()
    out.check()
    dh, _, tol = product(dy, w, bits)
    off(out.mid, *swiglu_back_of(dh, tol, gu))


@pytest.mark.parametrize("saved", [8, 16])
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,F,K", [
    (128, 128, 256), (1, 32, 64), (1, 1024, 2048), (3, 288, 576), (130, 416, 192), (515, 1024, 320),
    (33, 8192, 128), (700, 96, 4160), (64, 64, 16640)])
def test_backward(M, F, K, bits, saved):
    backward(M, F, K, bits, saved)


@pytest.mark.parametrize("saved", [8, 16])
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,F,K", [(2050, 1312, 448), (1031, 2720, 64), (2304, 2304, 1088), (300, 8192, 192)])
def test_backward_in_pairs(M, F, K, bits, saved):
    backward(M, F, K, bits, saved)


@pytest.mark.parametrize("M,F", [(9, 96), (2304, 2304)])
def test_backward_of_steep_gates(M, F):
    backward(M, F, 128, 8, 16, size=60.0)


def test_saved_zero_and_nan_scales():
    """A saved block of scale 0 stands for 2^-127 times its elements, one of 0xFF for NaN,
    in its own block only."""
    for M, F in ((70, 96), (2304, 2304)):
        dy, w = operand(M, 128, 8, 1), operand(F, 128, 8, 2)
        q, s = mx.cast_dim0(torch.randn(M, 2 * F, device="cuda").to(torch.bfloat16))
        at = blocked_at(M, 2 * F // 32, "cuda")
        want = mx.matmul_swiglu_backward(*dy, *w, (q, s))
        s[at[3, 0]], s[at[M - 1, F // 32 + 1]] = 0, 255
        got = mx.matmul_swiglu_backward(*dy, *w, (q, s))
        dh, _, tol = product(dy, w, 8)
        wanted, room = swiglu_back_of(dh, tol, mx_values(q, s))
        nan = torch.isnan(wanted)            # up's values reach dg alone
        assert torch.equal(torch.isnan(got), nan) and int(nan.sum()) == 32
        off(got[~nan], wanted[~nan], room[~nan])
        rest = torch.ones_like(got, dtype=torch.bool)
        rest[3, :32] = rest[3, F:F + 32] = False
        rest[M - 1, 32:64] = rest[M - 1, F + 32:F + 64] = False
        assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("M,F,K", [(96, 160, 192), (96, 256, 192), (2304, 1152, 256)])
def test_wrappers(M, F, K, bits):
    x, gate, up, h = forward(M, F, K, bits, False)
    w = tuple(zip(gate, up))
    assert torch.equal(mx.matmul_swiglu(*x, *w, bits=bits), h)
    h2, q, s = mx.matmul_swiglu(*x, *w, save=True, bits=bits)
    assert torch.equal(h2, h) and q.shape == (M, 2 * F)
    dy, w2 = operand(M, K, bits, 3), operand(F, K, bits, 4)
    d = mx.matmul_swiglu_backward(*dy, *w2, (q, s), bits=bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mx.matmul_swiglu(*x, *w, save=True, bits=bits, stream=side)
    back = mx.matmul_swiglu_backward(*dy, *w2, got[1:], bits=bits, stream=side)
    side.synchronize()
    for a, b in zip((*got, back), (h, q, s, d)):
        assert torch.equal(a, b)
    joint = torch.cat([gate[0], up[0]]), torch.cat([gate[1], up[1]])
    if F % 128:
        with pytest.raises(ValueError, match="apart"):
            mx.matmul_swiglu(*x, *joint, bits=bits)
        return
    for stream in (None, torch.cuda.current_stream()):
        assert torch.equal(mx.matmul_swiglu(*x, *joint, bits=bits, stream=stream), h)
    assert torch.equal(mx.matmul_swiglu(*x, [gate[0], up[0]], [gate[1], up[1]], bits=bits), h)


def test_offsets_past_32_bits():
    """131200 x 16640 gates and ups: saved bytes, h and gradients past 2^31 and 2^32, on
    sampled rows."""
    M, F, K = 131200, 16640, 64
    x, gate, up = operand(M, K, 8, 1), operand(F, K, 8, 2, 0.2), operand(F, K, 8, 3, 0.2)
    h, q, s = mx.matmul_swiglu(*x, *zip(gate, up), save=True)
    rows = torch.tensor([0, 1, 127, 64528, 64529, 65535, 65536, 129056, 129057, 131199], device="cuda")
    at = blocked_at(M, K // 32, "cuda")[rows]
    part = x[0][rows], mx.scales_to_blocked(x[1][at])
    pg, pu = product(part, gate, 8), product(part, up, 8)
    p, tol = torch.cat([pg[0], pu[0]], 1), torch.cat([pg[2], pu[2]], 1)
    off(h[rows], *swiglu_of(p, tol))
    del h
    saved_at = blocked_at(M, 2 * F // 32, "cuda")[rows]
    saved = q[rows].contiguous(), mx.scales_to_blocked(s[saved_at])
    check_saved(*saved, p, tol)
    d = mx.matmul_swiglu_backward(*x, *gate, (q, s))
    dh, _, tol = product(part, gate, 8)
    off(d[rows], *swiglu_back_of(dh, tol, mx_values(*saved)))
