"""What the build needs: libfa.so is built for users of the C library alone too, who
may have neither torch nor Python's headers."""
import os
import subprocess
import sys

import pytest

from exact_io_aware_96_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import os, subprocess, sys
{hide}
from exact_io_aware_96_b200 import build
ran = []
def run(cmd, **kw):
    ran.append(os.path.basename(cmd[0]))
    open(cmd[cmd.index("-o") + 1], "w").close()
    return subprocess.CompletedProcess(cmd, 0, "", "")
build.subprocess = type("Fake", (), dict(run=staticmethod(run)))
build.nvcc = lambda: "/opt/nvcc"
build.LIB, build.TORCH_LIB = (os.path.join(r"{at}", n) for n in ("libfa.so", "_fa_torch.so"))
build.build()
print(ran, sorted(os.listdir(r"{at}")))
"""
NO_TORCH = "sys.modules['torch'] = None"
NO_HEADERS = "import sysconfig; sysconfig.get_paths = lambda: dict(include='/nowhere')"


@pytest.mark.parametrize("hide", [NO_TORCH, NO_HEADERS], ids=["torch", "headers"])
def test_library_alone(tmp_path, hide):
    out = subprocess.run([sys.executable, "-c", PROGRAM.format(hide=hide, at=tmp_path)], cwd=ROOT, capture_output=True,
                         text=True, timeout=200)
    assert out.returncode == 0, out.stderr[-1500:]
    assert out.stdout.strip() == "['nvcc'] ['libfa.so']"
    assert "_fa_torch.so is not built" in out.stderr


def test_both(tmp_path):
    out = subprocess.run([sys.executable, "-c", PROGRAM.format(hide="", at=tmp_path)], cwd=ROOT, capture_output=True,
                         text=True, timeout=200)
    assert out.stdout.strip() == "['nvcc', 'g++'] ['_fa_torch.so', 'libfa.so']", out.stderr[-1500:]
    assert build.torch_missing() is None
