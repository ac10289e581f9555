"""Which kernel the plan sends the linear layer on 8-bit operands to (on the CPU: the
planner is plain C++).  The shapes are those whose results the GPU tests compare:
a change of the plan that leaves a kernel without a test shows here."""

import os
import shutil
import subprocess

import pytest

from linear_fp8_paths import PATHS
from means_nearest_centroid_amd import build as kbuild

TESTS = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("plan") / "linear_fp8_plan_print")
    res = subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I", kbuild.CSRC,
                          os.path.join(TESTS, "linear_fp8_plan_print.cpp"), "-o", exe],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return lambda *shape: subprocess.run([exe, *map(str, shape)], capture_output=True, text=True,
                                         check=True).stdout.split()


@pytest.mark.parametrize("N,D,F,half,single", PATHS)
def test_plan_of_the_tested_shapes(plan, N, D, F, half, single):
    assert plan(N, D, F) == [half, single]


def test_every_kernel_is_among_them():
    """Every tile shape, split and unsplit, with an odd and an even number of
    blocks of k where the kernel takes them in turns of two, and more than its
    stages hold."""
    for column, shapes in ((3, ("wide", "paired", "deep")), (4, ("paired", "deep"))):
        for shape in shapes:
            mine = [p[column].split(":") for p in PATHS if p[column].startswith(shape)]
            assert {int(s) > 1 for _, s, _ in mine} == {True, False}, shape
            assert {int(k) % 2 for _, _, k in mine} == {0, 1}, shape
            assert max(int(k) for _, _, k in mine) >= 8, shape
    cut = [p for p in PATHS if p[3].startswith("wide:1") and p[0] % 256 and p[2] % 8]
    assert cut and any(p[1] % 128 for p in cut)
