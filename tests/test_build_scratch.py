"""The build's check that the selective scan's kernels stay in their registers (a compiler's report; no compilation here)."""
import types

import pytest

from replayssm_persistent_rssm_amd import build

REPORT = """./scan_kernel.h:284:1: remark: Function Name: one [-Rpass-analysis=kernel-resource-usage]
./scan_kernel.h:284:1: remark:     VGPRs: 107 [-Rpass-analysis=kernel-resource-usage]
./scan_kernel.h:284:1: remark:     ScratchSize [bytes/lane]: 0 [-Rpass-analysis=kernel-resource-usage]
./scan_kernel.h:284:1: remark: Function Name: two [-Rpass-analysis=kernel-resource-usage]
./scan_kernel.h:284:1: remark:     ScratchSize [bytes/lane]: {} [-Rpass-analysis=kernel-resource-usage]
"""


@pytest.fixture()
def compiler(monkeypatch):
    """A compiler that prints what `said` holds; `asked` keeps its commands."""
    c = types.SimpleNamespace(said="", asked=[])

    def run(cmd, **kw):
        c.asked.append(cmd)
        return types.SimpleNamespace(returncode=0, stdout="", stderr=c.said)
    monkeypatch.setattr(build.subprocess, "run", run)
    return c


def test_every_scan_source_is_watched():
    assert set(build.NO_SCRATCH) == {s for s in build.SOURCES if s.startswith("rssm_inst_scan")}


@pytest.mark.parametrize("src", build.NO_SCRATCH)
def test_scratch_fails_the_build(compiler, src):
    compiler.said = REPORT.format(0)
    build._compile(src, False)
    assert "-Rpass-analysis=kernel-resource-usage" in compiler.asked[0]
    compiler.said = REPORT.format(44)
    with pytest.raises(RuntimeError, match=r"use scratch memory: two \(44 bytes a lane\)"):
        build._compile(src, False)
    compiler.said = ""
    with pytest.raises(RuntimeError, match="no resource report"):
        build._compile(src, False)


def test_other_sources_are_compiled_as_before(compiler):
    compiler.said = REPORT.format(44)
    build._compile("rssm_inst_f8.hip", False)
    assert not any("Rpass" in a for a in compiler.asked[0])
