"""The linear kernels' staging of unaligned rows reads nothing outside an
operand: its address arithmetic, which the kernels share with a program that
follows every run of it on the CPU."""

import os
import shutil
import subprocess

import pytest

from means_nearest_centroid_amd import build as kbuild

TESTS = os.path.dirname(os.path.abspath(__file__))


def test_no_run_leaves_its_operand(tmp_path):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "linear_staging_check")
    res = subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-I", kbuild.CSRC,
                          os.path.join(TESTS, "linear_staging_check.cpp"), "-o", exe],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stdout[-2000:]
    assert res.stdout.endswith("runs inside\n")
