"""The plan of the MX product, on the host: the cases of tests/mx_paths.py reach every kernel that it chooses."""
import math
import os
import random
import shutil
import subprocess

import pytest

from tests.mx_paths import CASES
from weight_only_int4_act_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))
# (kernel, 16-row fragments or rows / 64, bits, K cut into slices, tiles: K a multiple of 128)
PATHS = {("rows", rf, b, cut, None) for rf in (1, 2, 3, 4) for b in (8, 4) for cut in (False, True)} | {
    ("tile", wm, b, cut, whole) for wm in (1, 2, 4) for b in (8, 4) for cut in (False, True) for whole in (False, True)}


def paths(exe, cases):
    text = "".join("%d %d %d %d\n" % c for c in cases)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60).stdout.split("\n")
    got = [line.split() for line in out if line]
    assert len(got) == len(cases)
    return {(kind, int(size), c[3], int(nz) > 1, c[1] % 128 == 0 if kind == "tile" else None)
            for (kind, size, nz), c in zip(got, cases)}


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")):
        pytest.skip("needs hipcc")
    d = tmp_path_factory.mktemp("plan")
    exe = str(d / "mx_plan")
    r = subprocess.run([build.hipcc(), f"--offload-arch={build.ARCH}", "-O1", "-std=c++17", "-x", "hip",
                        os.path.join(HERE, "mx_plan.cpp"), "-x", "none", build.LIB, f"-Wl,-rpath,{build.PKG}", "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


def test_the_cases_reach_every_path(plan):
    assert paths(plan, [c + (b,) for c in CASES for b in (8, 4)]) == PATHS


def test_there_are_no_other_paths(plan):
    rng = random.Random(0)

    def size(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    cases = [(size(1, 70000), 32 * size(1, 4096), 8 * size(1, 16384), rng.choice((8, 4))) for _ in range(60000)]
    assert paths(plan, cases) <= PATHS
