"""A mode that watches what torch dispatches, as memory trackers do, sees the
wrappers' allocations."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import mxfp8_block_scaled_dim0_gb300 as mx

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()


class Dispatched(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.bytes = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        r = func(*args, **(kwargs or {}))
        if "empty" in str(func):
            self.bytes += r.nbytes
        return r


def calls():
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn((160, 96), generator=g, device="cuda").to(BF) for _ in range(2))
    gu = torch.randn((64, 128), generator=g, device="cuda").to(BF)
    w = torch.ones(96, device="cuda")
    _, mean, rstd = mx.layer_norm(x, w)
    a, b = mx.cast_dim0(x), mx.cast_dim0(dy)
    return {
        "cast 0": lambda: mx.cast_dim0(x),
        "cast 1": lambda: mx.cast_dim1(x),
        "cast both": lambda: mx.cast_dim0_dim1(x),
        "norm": lambda: mx.layer_norm(x, w, save=True),
        "norm back": lambda: mx.layer_norm_backward(dy, x, w, mean, rstd),
        "swiglu": lambda: mx.swiglu(gu, save=True),
        "swiglu back": lambda: (mx.swiglu_backward(gu[:, :64].contiguous(), gu),),
        "product": lambda: (mx.matmul(*a, *b),),
    }


def test_allocations_are_seen():
    for name, call in calls().items():
        want = call()
        with Dispatched() as seen:
            got = call()
        assert seen.bytes >= sum(t.nbytes for t in got), name
        for a, b in zip(got, want):
            assert torch.equal(a, b), name
