"""The build's steps: the C library needs hipcc alone, its torch binding comes after it.

Each test compiles one small source into a folder of its own; nothing in the tree changes.
"""
import os
import sys

import pytest

from conv2d_backward_amd import build


@pytest.fixture
def small_build(tmp_path, monkeypatch):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    monkeypatch.setattr(build, "SOURCES", ["noalloc.hip"])
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "binding.so"))
    return tmp_path


def test_library_is_built_without_torch(small_build, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)   # `import torch` raises ImportError
    assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)
    assert "torch" in capsys.readouterr().err


def test_library_is_linked_when_the_binding_fails(small_build, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError, match="seq_binding.cpp"):
        build.build()
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)
