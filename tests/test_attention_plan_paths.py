"""The plan of the attention over the cache, on the host: the cases of tests/attention_paths.py reach every kernel that it
chooses, and its workspace is the one that callers are told."""
import math
import os
import random
import shutil
import subprocess

import pytest

from tests.attention_paths import CASES
from weight_only_int4_act_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))
# (rows, numbers of a head, in slices)
PATHS = {(r, D, cut) for r in (16, 128, 256) for D in (64, 128) for cut in (False, True)} - {(256, 64, False)}


def paths(exe, cases):
    text = "".join("%d %d %d %d %d %d\n" % (B, n, -(-L // T) * T, Hq, Hk, D) for B, n, L, Hq, Hk, D, T in cases)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60).stdout.split("\n")
    got = [tuple(map(int, line.split())) for line in out if line]
    assert len(got) == len(cases)
    assert all(told for _, _, _, told in got), [c for c, g in zip(cases, got) if not g[3]][:4]
    assert all(rows * tiles >= c[1] * c[3] // c[4] for c, (rows, _, tiles, _) in zip(cases, got))
    return [(rows, c[5], split > 1) for (rows, split, _, _), c in zip(got, cases)]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")):
        pytest.skip("needs hipcc")
    exe = str(tmp_path_factory.mktemp("plan") / "attention_plan")
    r = subprocess.run([build.hipcc(), f"--offload-arch={build.ARCH}", "-O1", "-std=c++17", "-x", "hip",
                        os.path.join(HERE, "attention_plan.cpp"), "-x", "none", build.LIB, f"-Wl,-rpath,{build.PKG}", "-o", exe],
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

    heads = [(64, 8), (32, 8), (40, 8), (32, 32), (40, 40), (16, 1), (12, 4), (1, 1), (8, 2), (512, 4), (1024, 1024)]
    cases = []
    while len(cases) < 60000:
        Hq, Hk = rng.choice(heads)
        n, B, D = size(1, 9000), size(1, 600), rng.choice([64, 128])
        if n * B * (Hq + 2 * Hk) * D <= 1 << 31:
            cases.append((B, n, n + size(1, 100000), Hq, Hk, D, rng.choice([16, 32, 64, 128])))
    assert set(paths(plan, cases)) <= PATHS
