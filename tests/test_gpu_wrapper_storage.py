"""What the allocating wrappers return stands alone: every output has a storage of
its own, so that keeping, saving or freeing one does not do so to another."""
import io

import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.library()


def rnd(shape, seed, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def outputs():
    x, dy, w = rnd((160, 96), 1), rnd((160, 96), 2), rnd((96,), 3, torch.float32)
    gu = rnd((70, 256), 5)
    _, mean, rstd, q, s = mx.layer_norm(x, w, w, save=True)
    return {
        "norm": mx.layer_norm(x, w, w),
        "norm, save": mx.layer_norm(x, w, w, save=True),
        "norm back": mx.layer_norm_backward(dy, x, w, mean, rstd),
        "norm back, save": mx.layer_norm_backward(dy, (q, s), w, mean, rstd),
        "swiglu, save": mx.swiglu(gu, save=True),
        "cast 0": mx.cast_dim0(x),
        "cast 1": mx.cast_dim1(x),
        "cast both": mx.cast_dim0_dim1(x),
    }


def test_storages():
    for name, ts in outputs().items():
        assert len({t.untyped_storage().data_ptr() for t in ts}) == len(ts), name
        for t in ts:
            assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.nbytes, name


def test_scales_do_not_keep_the_bytes():
    x, w = rnd((4096, 4096), 1), rnd((4096,), 2, torch.float32)
    gu = rnd((2048, 4096), 3)
    for call, keep in ((lambda: mx.cast_dim0(x), 1), (lambda: mx.cast_dim1(x), 1),
                       (lambda: mx.cast_dim0_dim1(x), 3), (lambda: mx.swiglu(gu, save=True), 2),
                       (lambda: mx.layer_norm(x, w, save=True), 1),
                       (lambda: mx.layer_norm(x, w, save=True), 4)):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        kept = call()[keep]
        assert torch.cuda.memory_allocated() - before <= kept.nbytes + (2 << 20)


def test_saved_to_a_file_alone():
    _, s = mx.cast_dim0(rnd((1024, 1024), 1))
    f = io.BytesIO()
    torch.save(s, f)
    assert f.tell() < s.nbytes + 8192
