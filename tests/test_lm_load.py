"""CPU: the library loads where the CUDA runtime it was linked with is only torch's."""
import sys

import pytest

import stream_compaction_decoupled_gb300 as gb
from stream_compaction_decoupled_gb300 import _build


class Loader:
    """ctypes.CDLL, which fails until torch is there (its runtime would not be found)."""

    def __init__(self, whole, serves):
        self.whole, self.serves, self.calls = whole, serves, 0

    def __call__(self, path, *args, **kwargs):
        if path != gb.LIB_PATH:
            return self.whole(path, *args, **kwargs)
        self.calls += 1
        if not (self.serves and "torch" in sys.modules and self.calls > 1):
            raise OSError("libcudart.so.13: cannot open shared object file")
        return self.whole(path)


@pytest.mark.parametrize("serves", [True, False])
def test_torchs_runtime_serves(monkeypatch, serves):
    _build.build()
    loader = Loader(gb.ctypes.CDLL, serves)
    monkeypatch.setattr(gb, "_lib", None)
    monkeypatch.setattr(gb.ctypes, "CDLL", loader)
    if serves:
        assert gb.load().gb_version() > 0
    else:
        with pytest.raises(OSError):
            gb.load()
    assert loader.calls == 2
