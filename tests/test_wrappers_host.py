"""Loading of the binding with and without its compiled wrappers."""
import threading
import time

import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from mxfp8_block_scaled_dim0_gb300 import build as mxbuild


@pytest.fixture
def unloaded(monkeypatch):
    mxbuild.build()
    monkeypatch.setattr(mx, "_LIB", None)
    monkeypatch.setattr(mx, "_CALL", None)


def test_loads_without_the_compiled_wrappers(unloaded, monkeypatch, tmp_path):
    """The casts and operators need only the kernels' library: the checked functions
    serve, and say what is missing once."""
    x = torch.zeros(64, 96, dtype=torch.bfloat16)
    for content in (None, b"not a shared object"):
        path = tmp_path / ("absent.so" if content is None else "broken.so")
        if content is not None:
            path.write_bytes(content)
        monkeypatch.setattr(mx, "CALL_PATH", str(path))
        monkeypatch.setattr(mx, "_LIB", None)
        with pytest.warns(RuntimeWarning, match="compiled wrappers"):
            mx.library()
        assert mx._compiled("cast_dim0", x) is None
        for call in (lambda: mx.cast_dim0(x), lambda: mx.swiglu(x), lambda: mx.layer_norm(x, x[0])):
            with pytest.raises(ValueError, match="CUDA"):
                call()


def test_another_thread_sees_the_wrappers_with_the_library(unloaded, monkeypatch):
    """Two threads' first calls: neither finds the library before the wrappers."""
    load, failed = mx._load_call, []

    def slow():
        time.sleep(0.2)
        return load()

    def work():
        try:
            mx._compiled("cast_dim0", torch.zeros(64, 96, dtype=torch.bfloat16))
        except Exception as e:
            failed.append(e)

    monkeypatch.setattr(mx, "_load_call", slow)
    threads = [threading.Thread(target=work) for _ in range(2)]
    threads[0].start()
    time.sleep(0.1)
    threads[1].start()
    for t in threads:
        t.join()
    assert not failed, failed
