"""The allocating wrappers: the compiled ones and the checked path behind them give
the same results; outputs that share an allocation do not share bytes."""
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


def flat(r):
    return [r] if isinstance(r, torch.Tensor) else [t for t in r if t is not None]


def calls():
    x, dy, w, b = rnd((160, 96), 1), rnd((160, 96), 2), rnd((96,), 3, torch.float32), rnd((96,), 4, torch.float32)
    gu, dh = rnd((70, 256), 5), rnd((70, 128), 6)
    y, mean, rstd, q, s = mx.layer_norm(x, w, b, save=True)
    _, gq, gs = mx.swiglu(gu, save=True)
    a, c = mx.cast_dim0(x), mx.cast_dim0(dy)
    return {
        "norm": lambda: mx.layer_norm(x, w, b),
        "norm, bf16": lambda: mx.layer_norm(x, w.to(BF), b.to(BF)),
        "norm, no bias": lambda: mx.layer_norm(x, torch.nn.Parameter(w)),
        "norm, save": lambda: mx.layer_norm(x, w, b, save=True),
        "norm back": lambda: mx.layer_norm_backward(dy, x, w, mean, rstd),
        "norm back, save": lambda: mx.layer_norm_backward(dy, (q, s), w, mean, rstd),
        "norm back, no bias": lambda: mx.layer_norm_backward(dy, x, w, mean, rstd, bias=False),
        "swiglu": lambda: mx.swiglu(gu),
        "swiglu, save": lambda: mx.swiglu(gu, save=True),
        "swiglu back": lambda: mx.swiglu_backward(dh, gu),
        "swiglu back, save": lambda: mx.swiglu_backward(dh, (gq, gs)),
        "product": lambda: mx.matmul(*a, *c),
        "product, f32": lambda: mx.matmul(*a, *c, torch.float32),
        "product, float8": lambda: mx.matmul(a[0].view(torch.float8_e4m3fn), a[1], *c),
        "product, by column": lambda: mx.matmul(a[0].t().contiguous().t(), a[1], *c),
        "cast 0": lambda: mx.cast_dim0(x),
        "cast 1": lambda: mx.cast_dim1(x),
        "cast both": lambda: mx.cast_dim0_dim1(x),
    }


def test_compiled_and_checked_paths_agree(monkeypatch):
    for name, call in calls().items():
        taken = []
        compiled = mx._compiled

        def spy(*args):
            r = compiled(*args)
            taken.append(r is not None)
            return r

        monkeypatch.setattr(mx, "_compiled", spy)
        fast = flat(call())
        assert taken == [True], name
        monkeypatch.setattr(mx, "_compiled", lambda *args: None)
        slow = flat(call())
        monkeypatch.setattr(mx, "_compiled", compiled)
        assert len(fast) == len(slow), name
        for a, b in zip(fast, slow):
            assert a.dtype == b.dtype and a.shape == b.shape and a.device == b.device, name
            assert a.is_contiguous() and not a.requires_grad, name
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


def test_outputs_do_not_overlap():
    for name, call in calls().items():
        spans = sorted((t.data_ptr(), t.data_ptr() + t.nbytes) for t in flat(call()))
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:])), name
        assert all(lo % 256 == 0 for lo, _ in spans), name
        for t in flat(call()):
            end = t.storage_offset() * t.element_size() + t.nbytes
            assert end <= t.untyped_storage().nbytes(), name


def test_dropping_the_result_frees_the_activations():
    """What is saved for the backward pass does not keep the layer's output."""
    gu = rnd((4096, 4096), 1)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    h, q, s = mx.swiglu(gu, save=True)
    del h
    kept = torch.cuda.memory_allocated() - before
    assert kept <= q.nbytes + s.nbytes + (2 << 20)


def test_flags_of_other_types():
    x, w = rnd((64, 96), 1), rnd((96,), 2, torch.float32)
    assert len(mx.layer_norm(x, w, save=1)) == 5 and len(mx.layer_norm(x, w, None, 1, 0)) == 3
    assert len(mx.swiglu(rnd((64, 192), 3), save=1)) == 3
    _, mean, rstd = mx.layer_norm(x, w)
    assert mx.layer_norm_backward(x, x, w, mean, rstd, bias=0)[2] is None
    saved = list(mx.layer_norm(x, w, save=True)[3:])
    assert len(mx.layer_norm_backward(x, saved, w, mean, rstd)) == 3


def test_errors_carry_the_code():
    with pytest.raises(mx.MXError) as e:
        mx.swiglu(rnd((4, 96), 1), save=True)
    assert e.value.code == mx.MX_ERR_SHAPE
    with pytest.raises(mx.MXError) as e:
        mx.cast_dim1(rnd((33, 64), 1))
    assert e.value.code == mx.MX_ERR_SHAPE
    with pytest.raises(mx.MXError) as e:
        mx.layer_norm(rnd((8, 64), 1)[:, :].view(64, 8)[1:].reshape(63, 8), rnd((8,), 2, torch.float32), eps=float("nan"))
    assert e.value.code == mx.MX_ERR_SHAPE


def test_captured_in_a_graph():
    """Every call, in one graph: the same results from new contents of its inputs."""
    x, dy = rnd((160, 96), 1), rnd((160, 96), 2)
    w, gu, dh = rnd((96,), 3, torch.float32), rnd((160, 256), 5), rnd((160, 128), 6)

    def step():
        y, mean, rstd, q, s = mx.layer_norm(x, w, save=True)
        dx, dw, db = mx.layer_norm_backward(dy, (q, s), w, mean, rstd)
        h, gq, gs = mx.swiglu(gu, save=True)
        out = [y, mean, rstd, q, s, dx, dw, db, h, gq, gs, mx.swiglu_backward(dh, (gq, gs))]
        a, b = mx.cast_dim0(x), mx.cast_dim0(dy)
        return out + [mx.matmul(*a, *b), mx.matmul(*a, *b, torch.float32)]

    step()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = step()
    for t, seed in ((x, 11), (dy, 12), (gu, 13), (dh, 14)):
        t.copy_(rnd(tuple(t.shape), seed))
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, step()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
