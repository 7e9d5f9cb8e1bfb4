"""MX-FP4 casts and dequantisation on the GPU, every byte against the definition in 64
bits."""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from plain64 import blocked_at
from plain_fp4 import cast_rows, mx4_values

pytestmark = pytest.mark.gpu
GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()
    assert mx.mx_watchdog(clear=True) == 0
    yield
    torch.cuda.synchronize()
    assert mx.mx_watchdog(clear=True) == 0


def rnd(M, K, seed):
    """Values of uneven sizes with zeros and whole blocks of them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-20, 20, (M, K // 32, 1), generator=g, device="cuda").float()
                    ).expand(M, K // 32, 32).reshape(M, K)
    x[torch.rand(M, K, generator=g, device="cuda") < 0.05] = 0
    x[:, :32] *= (torch.rand(M, 1, generator=g, device="cuda") < 0.9).float()
    return x.to(torch.bfloat16)


class Buffer:
    """Bytes between guards."""

    def __init__(self, n):
        self.all = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.mid = self.all[GUARD:GUARD + n]

    def check(self):
        n = self.mid.numel()
        assert bool((self.all[:GUARD] == 0xA5).all()) and bool((self.all[GUARD + n:] == 0xA5).all())


def cast(x, dims):
    """{name: bytes} of a cast into guarded buffers."""
    M, K = x.shape
    size = {"q0": M * K // 2, "s0": mx.mx_blocked_bytes(M, K // 32), "q1": M * K // 2,
            "s1": mx.mx_blocked_bytes(K, M // 32)}
    names = [n for n in size if n[1] in dims]
    bufs = {n: Buffer(size[n]) for n in names}
    call = {"0": mx.mx_cast_fp4_dim0, "1": mx.mx_cast_fp4_dim1, "01": mx.mx_cast_fp4_dim0_dim1}[dims]
    call(x, *(bufs[n].mid for n in names))
    torch.cuda.synchronize()
    for b in bufs.values():
        b.check()
    return {n: b.mid for n, b in bufs.items()}


def check(x, dims):
    got = cast(x, dims)
    for d, y in (("0", x), ("1", x.t().contiguous())):
        if d in dims:
            q, s = cast_rows(y)
            assert torch.equal(got["s" + d], s), "scales of dim%s" % d
            assert torch.equal(got["q" + d].view(q.shape), q), "bytes of dim%s" % d


@pytest.mark.parametrize("M,K", [(1, 32), (1, 5120), (7, 96), (33, 160), (128, 128), (129, 224), (300, 256),
                                 (5, 288), (64, 1056), (1000, 512), (3, 16384), (4099, 64)])
def test_dim0(M, K):
    check(rnd(M, K, M + K), "0")


@pytest.mark.parametrize("dims", ["1", "01"])
@pytest.mark.parametrize("M,K", [(32, 32), (32, 160), (64, 96), (128, 128), (160, 64), (96, 1056),
                                 (1024, 512), (2080, 416), (640, 5120)])
def test_dim1_and_both(M, K, dims):
    check(rnd(M, K, M + K), dims)


def special():
    """Every finite bf16 magnitude at some place of blocks whose largest value varies, both
    signs; subnormals; zeros of both signs; Inf and NaN blocks."""
    bits = torch.arange(0, 0x7F80, device="cuda").to(torch.int16)
    v = bits.view(torch.bfloat16).float()
    sign = torch.where(torch.arange(v.numel(), device="cuda") % 3 == 0, -1.0, 1.0)
    rows = [(v * sign)[: v.numel() // 1024 * 1024].reshape(-1, 1024)]
    # Mantissas of bf16 at every exponent distance from the block's largest value.
    m = 1 + torch.arange(128, device="cuda").float() / 128
    for top in (0, 30, -100, 120):
        for down in range(0, 7):
            b = (m * 2.0 ** (top - down)).reshape(-1, 8).repeat(1, 4)[:, :32].clone()
            b[:, 0] = 2.0 ** top
            rows.append(torch.cat([b, -b], 1).repeat(1, 16))
    z = torch.zeros(8, 1024, device="cuda")
    z[1] = -0.0
    z[2, ::7] = float("inf")
    z[3, 5::64] = float("nan")
    z[4, ::32] = -float("inf")
    z[5] = 2.0 ** -133
    z[6, ::2] = -(2.0 ** -130)
    z[7, 3::32] = torch.finfo(torch.bfloat16).max
    x = torch.cat(rows + [z]).to(torch.bfloat16)
    pad = -x.shape[0] % 32
    return torch.cat([x, torch.zeros(pad, 1024, device="cuda", dtype=torch.bfloat16)])


def test_special_values():
    x = special()
    check(x, "0")
    check(x, "01")
    check(x.t().contiguous(), "1")


def test_wrappers_and_their_types():
    x = rnd(96, 192, 3)
    q0, s0, q1, s1 = mx.cast_fp4_dim0_dim1(x)
    assert q0.shape == (96, 96) and q1.shape == (192, 48) and q0.dtype == torch.uint8
    for a, b in zip(mx.cast_fp4_dim0(x) + mx.cast_fp4_dim1(x), (q0, s0, q1, s1)):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mx.cast_fp4_dim0_dim1(x, stream=side)
    back = mx.dequant_fp4(got[0], got[1], stream=side)
    side.synchronize()
    assert torch.equal(got[0], q0) and torch.equal(got[3], s1)
    assert torch.equal(back, mx.dequant_fp4(q0, s0))
    if hasattr(torch, "float4_e2m1fn_x2"):
        assert torch.equal(mx.dequant_fp4(q0.view(torch.float4_e2m1fn_x2), s0), back)


@pytest.mark.parametrize("R,C", [(1, 32), (3, 96), (17, 256), (130, 288), (515, 2720), (64, 8192), (2, 16416),
                                 (5000, 64)])
def test_dequant(R, C):
    g = torch.Generator(device="cuda").manual_seed(R + C)
    q = torch.randint(0, 256, (R, C // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.full((mx.mx_blocked_bytes(R, C // 32),), 255, dtype=torch.uint8, device="cuda")
    at = blocked_at(R, C // 32, "cuda")
    s[at] = torch.randint(0, 256, at.shape, generator=g, device="cuda").to(torch.uint8)
    buf = Buffer(2 * R * C)
    out = buf.mid.view(torch.bfloat16).view(R, C)
    mx.mx_dequant_fp4(q, s, out)
    torch.cuda.synchronize()
    buf.check()
    want = mx4_values(q, s).to(torch.bfloat16)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(out), nan)
    assert torch.equal(out.view(torch.int16)[~nan], want.view(torch.int16)[~nan])


def test_every_code_and_scale():
    q = torch.arange(256, device="cuda", dtype=torch.uint8)[None, :16].repeat(4096, 1)
    q = (q + 16 * (torch.arange(4096, device="cuda", dtype=torch.int64) % 16)[:, None]).to(torch.uint8)
    s = torch.zeros(mx.mx_blocked_bytes(4096, 1), dtype=torch.uint8, device="cuda")
    s[blocked_at(4096, 1, "cuda")] = (torch.arange(4096, device="cuda") // 16).to(torch.uint8)[:, None]
    out, want = mx.dequant_fp4(q, s), mx4_values(q, s).to(torch.bfloat16)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(out), nan)
    assert torch.equal(out.view(torch.int16)[~nan], want.view(torch.int16)[~nan])


def test_round_trip_of_its_own_values():
    """A cast of values that MX-FP4 can hold is exact, and one of its results repeats it."""
    x = rnd(256, 512, 9)
    q, s = mx.cast_fp4_dim0(x)
    y = mx.dequant_fp4(q, s)
    assert torch.equal(mx.dequant_fp4(*mx.cast_fp4_dim0(y)), y)


def test_offsets_past_32_bits():
    """65536 x 65536 values: bytes, scales and inputs past 2^31 and 2^32, on sampled rows."""
    n = 65536
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(n, n, dtype=torch.bfloat16, device="cuda")
    for i in range(0, n, 8192):
        x[i:i + 8192] = torch.randn(8192, n, generator=g, device="cuda", dtype=torch.bfloat16)
    q0, s0, q1, s1 = mx.cast_fp4_dim0_dim1(x)
    rows = torch.tensor([0, 1, 127, 128, 32767, 32768, 65407, 65535], device="cuda")
    at = blocked_at(n, n // 32, "cuda")[rows]
    for q, s, part in ((q0, s0, x[rows]), (q1, s1, x[:, rows].t().contiguous())):
        want_q, want_s = cast_rows(part)
        assert torch.equal(q[rows], want_q)
        assert torch.equal(s[at], want_s[blocked_at(8, n // 32, "cuda")])
    a, b = mx.cast_fp4_dim0(x)
    assert torch.equal(a, q0) and torch.equal(b, s0)
    del x, q1, s1, a, b
    out = mx.dequant_fp4(q0, s0)
    want = torch.cat([mx4_values(q0[r:r + 1], mx.scales_to_blocked(s0[at[i:i + 1]]))
                      for i, r in enumerate(rows.tolist())])
    assert torch.equal(out[rows], want.to(torch.bfloat16))
