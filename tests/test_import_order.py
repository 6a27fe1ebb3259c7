"""The package and torch in one process use one HIP runtime, whichever is imported first."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import importlib
for name in {order!r}:
    importlib.import_module(name)
paths = {{line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line}}
assert len(paths) == 1, paths
{more}
"""

PACKAGE = "replayssm_persistent_rssm_amd"


def run(order, more=""):
    subprocess.run([sys.executable, "-c", CODE.format(order=order, more=more)], cwd=ROOT, check=True, timeout=300)


@pytest.mark.parametrize("order", [(PACKAGE, "torch"), ("torch", PACKAGE)])
def test_one_runtime(order):
    run(order)


@pytest.mark.gpu
def test_a_call_after_the_package_came_first():
    run((PACKAGE, "torch"), f"""
import torch, {PACKAGE} as rp
x, w, s = torch.ones(3, 8, device="cuda"), torch.ones(4, 8, device="cuda"), torch.zeros(1, 3, 8, device="cuda")
y, i = torch.empty_like(x), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
rp.rssm_causal_conv(x, w, y, s, i[:1], i, silu=False)
assert y[:, 0].tolist() == [1.0, 2.0, 3.0]
""")
