"""The build: the C library alone where torch is missing, and no binding that was compiled
against another Python or torch."""
import os
import sys
import sysconfig

import pytest

from activation_sparse_gemm_lynx_b200 import build, lynx


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


def test_a_binding_for_another_torch_is_not_used(monkeypatch, recorded):
    import torch

    build.build(force=False)
    assert build.binding_up_to_date() or recorded  # here as built, or asked for
    del recorded[:]
    here = build.binding_path()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert build.binding_path() != here and not build.binding_up_to_date()
    build.build()
    assert recorded[-1:] == ["binding"]
    monkeypatch.setattr(lynx, "_compiled", None)
    monkeypatch.setattr(lynx, "library", lambda: None)
    with pytest.raises(ImportError, match="build"):
        lynx.lynx_ckpt8_store(None)


def test_a_binding_for_another_python_is_not_used(monkeypatch):
    here = build.binding_path()
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-399" if n == "SOABI" else real(n))
    assert build.binding_path() != here and not build.binding_up_to_date()
