"""The build: the C library alone where torch is missing."""
import os
import sys
import sysconfig

import pytest

from activation_sparse_gemm_lynx_b200 import build


@pytest.fixture
def recorded(monkeypatch):
    """build() with its two compilers replaced by a list of what they were asked for."""
    calls = []
    monkeypatch.setattr(build, "build_library", lambda verbose=False: calls.append("library"))
    monkeypatch.setattr(build, "build_binding", lambda: calls.append("binding"))
    return calls


def test_both_are_built(recorded):
    assert build.build(force=True) == build.LIB
    assert recorded == ["library", "binding"]


def test_without_torch_the_c_library_is_built(monkeypatch, recorded, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    assert build.build(force=True) == build.LIB
    assert recorded == ["library"]
    assert "torch" in capsys.readouterr().err


def test_without_python_headers_the_c_library_is_built(monkeypatch, recorded, capsys, tmp_path):
    paths = {**sysconfig.get_paths(), "include": os.fspath(tmp_path)}
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    assert build.build(force=True) == build.LIB
    assert recorded == ["library"]
    assert "headers" in capsys.readouterr().err
