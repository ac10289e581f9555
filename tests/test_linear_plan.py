"""Which kernel the linear operators' plan sends a shape to (on the CPU: the
planner is plain C++).  The shapes are those whose results the GPU tests
compare: a change of the plan that leaves a kernel without a test shows
here."""

import os
import shutil
import subprocess

import pytest

from linear_paths import PATHS
from means_nearest_centroid_amd import build as kbuild

TESTS = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("plan") / "linear_plan_print")
    res = subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I", kbuild.CSRC,
                          os.path.join(TESTS, "linear_plan_print.cpp"), "-o", exe],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return lambda *shape: subprocess.run([exe, *map(str, shape)], capture_output=True, text=True,
                                         check=True).stdout.split()


@pytest.mark.parametrize("N,D,F,extra,forward,dx,dw", PATHS)
def test_plan_of_the_tested_shapes(plan, N, D, F, extra, forward, dx, dw):
    assert plan(N, D, F, extra) == [forward, dx, dw]


@pytest.mark.parametrize("N,D,F", [(1, 4096, 4096), (16, 515, 1001)])
def test_few_rows_have_a_kernel_of_their_own(plan, N, D, F):
    assert plan(N, D, F, 0)[0].startswith("rows:")


def test_every_kernel_is_among_them():
    """The forward product and both gradients of every tile shape, with enough
    tiles of k for the pipelined loop (2 S for S stages, and the last one left
    out for unaligned rows), and split ones of the shapes that the plan splits."""
    for column in (4, 5, 6):
        long = {p[column].split(":")[0].rstrip("*") for p in PATHS
                if int(p[column].split(":")[2]) >= (8 if p[column].startswith("deep") else 5)}
        assert {"wide", "paired", "deep", "unaligned"} <= long, column
        split = {p[column].split(":")[0] for p in PATHS if int(p[column].split(":")[1]) > 1}
        assert {"deep", "unaligned"} <= split, column
