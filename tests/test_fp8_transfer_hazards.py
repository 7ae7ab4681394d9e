"""What the inline assembly of the 8-bit product's tile kernels relies on, read from their assembly as both libraries' flags
make it: the checks of tests/test_mx_transfer_hazards.py on these kernels."""
import os
import shutil
import subprocess

import pytest

from tests.test_mx_accumulators import _functions
from tests.test_mx_transfer_hazards import _check
from weight_only_int4_act_amd import build


@pytest.mark.skipif(not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")), reason="needs hipcc")
@pytest.mark.parametrize("extra", [[], ["-DAWQ_LDS_POISON"]], ids=["library", "lds_poison"])
def test_what_the_assembly_relies_on(tmp_path, extra):
    out = str(tmp_path / "gemm.s")
    subprocess.run([build.hipcc(), *build.FLAGS, *extra, "--cuda-device-only", "-S",
                    os.path.join(build.CSRC, "awq_fp8_gemm.hip"), "-o", out], check=True, capture_output=True)
    with open(out) as f:
        kernels = _functions(f.read().replace("k_fp8_gemm_tile", "k_mx_gemm_tile"))   # the name that it looks for
    assert len(kernels) == 6
    for name, code in kernels.items():
        products, transfers, bad = _check(code)
        assert products >= 8 and transfers >= 16 and not bad, (name, bad[:4])
