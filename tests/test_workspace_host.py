"""The per-stream workspace's host code against a model of the allocator: no
GPU, no HIP runtime call (the test program defines those it needs)."""

import os
import shutil
import subprocess

import pytest

from means_nearest_centroid_amd import build as kbuild

TESTS = os.path.dirname(os.path.abspath(__file__))


def test_workspace_of_captured_calls(tmp_path):
    if shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "workspace_check")
    cmd = [kbuild.hipcc(), f"--offload-arch={kbuild.ARCH}", "-O1", "-std=c++17",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-x", "hip",
           "-I", kbuild.INCLUDE, "-I", kbuild.CSRC,
           os.path.join(TESTS, "workspace_check.cpp"),
           os.path.join(kbuild.CSRC, "kmeans_workspace.hip"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout[-2000:]
