"""The counting of shared items (csrc/join_rule.h) over every order of the CTAs: each share is joined exactly once,
whoever begins late, and a wait for a count that never comes in ends within its limit."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "int4_weight_only_affine_gb300", "csrc")


def test_every_share_is_joined_once(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    exe = str(tmp_path / "join_orders")
    subprocess.run([cxx, "-std=c++17", "-O2", "-I" + CSRC, os.path.join(ROOT, "tests", "join_orders.cpp"), "-o", exe],
                   check=True, timeout=120)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout
