"""The plan of the product with scales per 128, on the host: the cases of tests/fp8_paths.py reach every kernel that it
chooses."""
import math
import os
import random
import shutil
import subprocess

import pytest

from tests.fp8_paths import CASES
from weight_only_int4_act_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))
# (kernel, 16-row fragments or rows / 64, K cut into slices, tiles: K a multiple of 128)
PATHS = {("rows", rf, cut, None) for rf in (1, 2, 4) for cut in (False, True)} | {
    ("tile", wm, cut, whole) for wm in (1, 2, 4) for cut in (False, True) for whole in (False, True)}


def paths(exe, cases):
    text = "".join("%d %d %d\n" % c for c in cases)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60).stdout.split("\n")
    got = [line.split() for line in out if line]
    assert len(got) == len(cases)
    return [(kind, int(size), int(nz) > 1, c[1] % 128 == 0 if kind == "tile" else None)
            for (kind, size, nz), c in zip(got, cases)]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")):
        pytest.skip("needs hipcc")
    exe = str(tmp_path_factory.mktemp("plan") / "fp8_plan")
    r = subprocess.run([build.hipcc(), f"--offload-arch={build.ARCH}", "-O1", "-std=c++17", "-x", "hip",
                        os.path.join(HERE, "fp8_plan.cpp"), "-x", "none", build.LIB, f"-Wl,-rpath,{build.PKG}", "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


def test_the_cases_reach_every_path_once(plan):
    got = paths(plan, CASES)
    assert set(got) == PATHS and len(got) == len(PATHS)


def test_there_are_no_other_paths(plan):
    rng = random.Random(0)

    def size(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    cases = [(size(1, 70000), 16 * size(1, 4096), 8 * size(1, 16384)) for _ in range(60000)]
    assert set(paths(plan, cases)) <= PATHS
