"""The build of the library and of the compiled binding (CPU only)."""
import importlib
import os

import pytest
import torch

f = pytest.importorskip("fp8_kv_cache_quant_gb300")
b = importlib.import_module("fp8_kv_cache_quant_gb300.build")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree of one small kernel, built into a folder of its own."""
    (tmp_path / "small.cu").write_text('extern "C" int fkv_small() { return 7; }\n')
    (tmp_path / "binding.cpp").write_text("int x;\n")
    for name in ("PKG", "CSRC", "BUILD_DIR"):
        monkeypatch.setattr(b, name, str(tmp_path))
    monkeypatch.setattr(b, "OUT", str(tmp_path / "libfp8kv.so"))
    monkeypatch.setattr(b, "SOURCES", ["small.cu"])
    return tmp_path


def test_the_library_does_not_need_the_binding(tree, monkeypatch):
    monkeypatch.setenv("CXX", "/bin/false")              # no compiler for Python's and torch's headers
    assert b.build(library_only=True) == b.OUT and os.path.exists(b.OUT)
    os.remove(b.OUT)
    with pytest.raises(RuntimeError, match="is built, the compiled binding is not"):
        b.build()
    assert os.path.exists(b.OUT) and not os.path.exists(b.binding_path())


def test_the_binding_belongs_to_one_python_and_one_torch(tree, monkeypatch):
    here = b.binding_path()
    assert torch.__version__ in os.path.basename(here) and "cpython-3" in os.path.basename(here)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert b.binding_path() != here and b._stale(b.binding_path(), ["binding.cpp"])
    monkeypatch.setattr(f, "_compiled", None)
    monkeypatch.setattr(f, "load_library", lambda: None)
    with pytest.raises(RuntimeError, match="0.0.1.* not built"):
        f.load_binding()
