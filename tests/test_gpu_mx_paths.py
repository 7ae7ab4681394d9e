"""The MX product on the GPU in every kernel that its plan chooses: against float64, and on the LDS-poison debug
build (a child process, because the binding loads one library per process)."""
import os
import subprocess
import sys

import pytest

from tests.mx_paths import CASES
from tests.mx_util import check_product, product, random_acts, random_weights

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "weight_only_int4_act_amd", "libawq_ldspoison.so")


def case(M, K, N, bits):
    xc, xs, x = random_acts(M, K, bits, M + K + N)
    wc, wsc, w = random_weights(K, N, M + K + N + 1)
    check_product(product(xc, xs, wc, wsc, M, K, N), x, w, bits, (M, K, N, bits))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,K,N", CASES)
def test_product_on_every_path(M, K, N, bits):
    case(M, K, N, bits)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_every_path_under_lds_poison(bits):
    assert os.path.exists(LIB), f"{LIB} is missing: build with `python -m weight_only_int4_act_amd.build`"
    r = subprocess.run([sys.executable, "-u", os.path.abspath(__file__), str(bits)], capture_output=True, text=True,
                       env={**os.environ, "AWQ_LIBRARY": LIB, "PYTHONPATH": ROOT}, timeout=110)
    print(r.stdout[-4000:])
    assert r.returncode == 0 and "[poison] all paths ok" in r.stdout, f"{r.stdout[-2000:]}\n{r.stderr[-4000:]}"


if __name__ == "__main__":
    for size in CASES:
        print("[poison] product", *size, sys.argv[1], flush=True)
        case(*size, int(sys.argv[1]))
    print("[poison] all paths ok", flush=True)
