"""Loading of the binding with and without its compiled wrappers."""
import os
import subprocess
import sys
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


OTHER_TORCH = """
import subprocess, warnings
import torch
torch.__version__ = torch.torch_version.TorchVersion("9.9.9")
import mxfp8_block_scaled_dim0_gb300 as mx
from mxfp8_block_scaled_dim0_gb300 import build
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    mx.library()
assert mx._CALL is None and len(seen) == 1, seen
ran = []
def run(cmd, **kwargs):
    ran.append(cmd)
    return subprocess.CompletedProcess(cmd, 1, "", "not run")
build.subprocess.run = run
try:
    build.build_call()
except RuntimeError as e:
    assert "not run" in str(e)
assert len(ran) == 1, ran
"""


def test_wrappers_of_another_torch_are_neither_loaded_nor_kept():
    """They are compiled against one torch's classes: under another they are built
    anew, and until then not loaded."""
    mxbuild.build()
    r = subprocess.run([sys.executable, "-c", OTHER_TORCH], cwd=os.path.dirname(mxbuild.PKG),
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
