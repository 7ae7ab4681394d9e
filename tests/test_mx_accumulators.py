"""The tile kernels of the MX product write their matrix-core instructions as inline assembly, which the
compiler's hazard recogniser does not see.  Their assembly, as the library's own flags make it: on no path is an
accumulation register read or copied after a product without the settling wait between, and none is written
within two instructions before a product."""
import os
import re
import shutil
import subprocess

import pytest

from weight_only_int4_act_amd import build

FAR = 99
SETTLE = {8: 12, 4: 8}      # wait states that the compiler itself leaves after a product, by the activations' bits


def _functions(text):
    """{name: instructions}; an instruction is (mnemonic, operands), a label (None, name)."""
    out, name = {}, None
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        if m := re.match(r"(_Z\w*k_mx_gemm_tile\w*):$", line):
            name = m.group(1)
            out[name] = []
        elif line.startswith(".end_amdhsa_kernel") or line.startswith(".section"):
            name = None
        elif name and (m := re.match(r"(\.L\w+):$", line)):
            out[name].append((None, m.group(1)))
        elif name and line and not line.startswith((".", "#")):
            op, _, rest = line.partition(" ")
            out[name].append((op, rest))
    return out


def _successors(code, labels, i):
    op, rest = code[i]
    if op == "s_endpgm":
        return []
    if op == "s_branch":
        return [labels[rest.strip()]]
    if op and op.startswith("s_cbranch"):
        return [labels[rest.strip()], i + 1]
    return [i + 1] if i + 1 < len(code) else []


def _check(code, settle):
    """(products, offences): states (product in flight, instructions since a write of an accumulator)."""
    labels = {rest: i for i, (op, rest) in enumerate(code) if op is None}
    seen, todo, bad = {}, [(0, False, FAR)], set()
    while todo:
        i, hot, since = todo.pop()
        old = seen.get(i)
        if old is not None:
            hot, since = hot or old[0], min(since, old[1])
            if (hot, since) == old:
                continue
        seen[i] = (hot, since)
        op, rest = code[i]
        if op is not None:
            wait = int(rest) + 1 if op == "s_nop" else 1
            if op.startswith("v_mfma"):
                if since < 2:
                    bad.add((i, "written right before", op, rest))
                hot, since = True, min(since + 1, FAR)
            else:
                if hot and op == "s_nop" and wait >= settle:
                    hot = False
                first, _, others = rest.partition(",")
                acc = re.compile(r"\ba(\d|\[)")
                stores = "store" in op
                if hot and acc.search(rest if stores else others):
                    bad.add((i, "read in flight", op, rest))
                since = 0 if acc.search(first) and not stores else min(since + wait, FAR)
        todo += [(j, hot, since) for j in _successors(code, labels, i)]
    return sum(op is not None and op.startswith("v_mfma") for op, _ in code), sorted(bad)


@pytest.mark.skipif(not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")), reason="needs hipcc")
def test_accumulators_are_settled(tmp_path):
    out = str(tmp_path / "gemm.s")
    subprocess.run([build.hipcc(), *build.FLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, "awq_mx_gemm.hip"),
                    "-o", out], check=True, capture_output=True)
    with open(out) as f:
        kernels = _functions(f.read())
    assert len(kernels) == 12
    for name, code in kernels.items():
        products, bad = _check(code, SETTLE[8 if "ILi8E" in name else 4])
        assert products >= 64 and not bad, (name, bad[:4])


def test_the_check_sees_mistakes():
    mfma = ("v_mfma_scale_f32_16x16x128_f8f6f4", "a[0:3], v[0:3], v[4:7], a[0:3], v8, v9")
    read, write, end = ("v_accvgpr_read_b32", "v0, a1"), ("v_accvgpr_write_b32", "a1, v0"), ("s_endpgm", "")
    wait = ("s_nop", "15")
    assert not _check([mfma, wait, read, end], 16)[1] and _check([mfma, wait, read, end], 17)[1]
    assert _check([mfma, read, end], 8)[1]
    assert _check([mfma, ("buffer_store_dwordx4", "a[0:3], v1, s[0:3], 0 offen"), end], 8)[1]
    assert _check([write, mfma, end], 8)[1] and not _check([write, ("s_nop", "1"), mfma, end], 8)[1]
    loop = [(None, ".L1"), read, mfma, ("s_cbranch_scc1", ".L1"), wait, end]
    assert _check(loop, 8)[1] and not _check(loop[:3] + [wait] + loop[3:], 8)[1]
