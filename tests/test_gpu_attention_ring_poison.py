"""Race test of the attention's tiles: the cases of tests/attention_ring_poison_cases.py against the LDS-poison debug build, in
a child process (the binding loads one library per process)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "weight_only_int4_act_amd", "libawq_ldspoison.so")


@pytest.mark.gpu
def test_tiles_under_lds_poison():
    assert os.path.exists(LIB), f"{LIB} is missing: build with `python -m weight_only_int4_act_amd.build`"
    r = subprocess.run([sys.executable, "-u", os.path.join(ROOT, "tests", "attention_ring_poison_cases.py")],
                       capture_output=True, text=True, env={**os.environ, "AWQ_LIBRARY": LIB}, timeout=110)
    print(r.stdout[-4000:])
    assert r.returncode == 0 and "[poison] all cases ok" in r.stdout, f"{r.stdout[-2000:]}\n{r.stderr[-4000:]}"
