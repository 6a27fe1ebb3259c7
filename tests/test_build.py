"""The build where parts of the usual machine are missing (no compilation here)."""
import os
import sys

import pytest


@pytest.fixture()
def build(monkeypatch, tmp_path):
    from replayssm_persistent_rssm_amd import build
    monkeypatch.setattr(build, "FAST_PATH", str(tmp_path / "_fast_calls.so"))
    return build


def test_libraries_build_without_torch(build, monkeypatch, capsys):
    """The C libraries need no torch: only the binding's extension is left out, with a note."""
    monkeypatch.setattr(build, "_compile", lambda src, verbose: src)
    linked = []
    monkeypatch.setattr(build, "_link", lambda objs, path, verbose: linked.append((len(objs), path)))
    monkeypatch.setitem(sys.modules, "torch", None)          # an import raises ImportError
    assert build.build() == build.LIB_PATH
    assert linked == [(len(build.SOURCES), build.LIB_PATH), (len(build.POOL_SOURCES), build.POOL_LIB_PATH)]
    assert "left out" in capsys.readouterr().err and not os.path.exists(build.FAST_PATH)


def test_host_compiler(build, monkeypatch):
    monkeypatch.setenv("CXX", "my-c++")
    assert build._cxx() == "my-c++"
    monkeypatch.delenv("CXX")
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    assert build._cxx() == os.path.join(os.path.dirname(build.HIPCC), "amdclang++")
