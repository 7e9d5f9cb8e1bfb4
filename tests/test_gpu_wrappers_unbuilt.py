"""Where the compiled wrappers are not built, every allocating wrapper works all the
same."""
import pytest
import torch

import mxfp8_block_scaled_dim0_gb300 as mx
from test_gpu_wrappers import calls, flat

pytestmark = pytest.mark.gpu


def test_same_results(monkeypatch, tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    want = {name: flat(call()) for name, call in calls().items()}
    monkeypatch.setattr(mx, "_LIB", None)
    monkeypatch.setattr(mx, "_CALL", None)
    monkeypatch.setattr(mx, "CALL_PATH", str(tmp_path / "absent.so"))
    with pytest.warns(RuntimeWarning, match="compiled wrappers"):
        mx.library()
    for name, call in calls().items():
        got = flat(call())
        assert len(got) == len(want[name]), name
        for a, b in zip(got, want[name]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
