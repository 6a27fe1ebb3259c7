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


def test_the_named_build_command_needs_no_built_library(monkeypatch):
    """What the message about a missing library says can be run there: the package itself cannot be
    imported yet, so the command may not go through it."""
    import re
    import subprocess

    import replayssm_persistent_rssm_amd._binding as b
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    monkeypatch.setattr(b, "LIB_PATH", "/nowhere/lib.so")
    with pytest.raises(ImportError) as e:
        b._load()
    script = re.search(r"`python (\S+\.py)`", str(e.value)).group(1)
    code = "import runpy, sys; runpy.run_path(sys.argv[1], run_name='x'); assert 'replayssm_persistent_rssm_amd' not in sys.modules"
    subprocess.run([sys.executable, "-c", code, script], cwd=root, check=True)
