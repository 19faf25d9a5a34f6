"""The table of shared-memory limits (csrc/smem_limits.h) under a host compiler: one entry for a kernel on a device
whatever sizes it takes, and no limit that is ever lowered, also past the table's last entry."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "int4_weight_only_affine_gb300", "csrc")


def test_limits_are_only_raised(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    exe = str(tmp_path / "smem_limits")
    subprocess.run([cxx, "-std=c++17", "-O2", "-pthread", "-I" + CSRC, os.path.join(ROOT, "tests", "smem_limits.cpp"), "-o", exe],
                   check=True, timeout=120)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
