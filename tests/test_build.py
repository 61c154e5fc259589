"""What is built when: the delta rule's calls and the C library need nvcc alone, the operators of layer.py a C++
compiler and Python's headers too."""
import pytest
import torch

import fp8_state_qat_gb300 as lib
from fp8_state_qat_gb300 import build, gdnqat, layer


@pytest.fixture
def no_compiler(monkeypatch, tmp_path):
    """No extension is there, and none can be compiled; the library has not been loaded yet."""
    lib.load()

    def fails(*a):
        raise RuntimeError("g++ failed on layer_ext.cpp: no Python.h")
    monkeypatch.setattr(build, "EXT_PATH", str(tmp_path / "gdnqat_layer.so"))
    monkeypatch.setattr(build, "compile_extension", fails)
    monkeypatch.setattr(gdnqat, "_lib", None)


def test_library_loads_without_the_extension(no_compiler):
    assert lib.load() is not None
    assert lib.chunk_workspace_bytes((1, 64, 1, 64), (1, 64, 1, 64)) > 0


def test_layer_operators_say_what_is_missing(no_compiler, monkeypatch):
    monkeypatch.setattr(layer, "_ext", layer._Unloaded())
    t = torch.zeros(2, 8)
    with pytest.raises(RuntimeError, match="layer_ext"):
        lib.gated_norm_fwd(t, t, t[0])
