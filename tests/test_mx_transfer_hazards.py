"""What the inline assembly of the MX product's tile kernels relies on and the compiler does not see, read from their
assembly as the library's own flags make it (both libraries'):
  - M0, the LDS address of a transfer, is written by each transfer for itself, one wait state before its use, and by
    nothing else;
  - no vector instruction writes an element or scale of a product within two wait states before it;
  - no vector instruction writes a scalar register within five wait states before a transfer that reads it."""
import os
import re
import shutil
import subprocess

import pytest

from tests.test_mx_accumulators import _functions, _successors
from weight_only_int4_act_amd import build

VGPR_STATES, SGPR_STATES = 2, 5


def _registers(text):
    """{('v' | 's', number)} of an operand list."""
    out = set()
    for kind, a, b in re.findall(r"\b([vs])\[(\d+):(\d+)\]", text):
        out |= {(kind, n) for n in range(int(a), int(b) + 1)}
    return out | {(kind, int(n)) for kind, n in re.findall(r"\b([vs])(\d+)\b", text)}


def _vector_writes(op, rest):
    """Registers that a vector-ALU instruction writes (its first operand; the second too where it is a mask or swapped)."""
    if not op.startswith("v_") or op.startswith("v_mfma"):
        return set()
    operands = re.split(r",\s*", rest)
    out = _registers(operands[0])
    if "_swap" in op or "_co_" in op or "div_scale" in op:
        out |= _registers(operands[1])
    return out


def _is_transfer(op, rest):
    return op.startswith("buffer_load") and re.search(r"\blds\b", rest)


def _check(code):
    """(products, transfers, offences)."""
    labels = {rest: i for i, (op, rest) in enumerate(code) if op is None}
    bad, products, transfers = [], 0, 0
    for i, (op, rest) in enumerate(code):
        if op is None:
            continue
        products += op.startswith("v_mfma")
        if _is_transfer(op, rest):
            transfers += 1
            own = i > 1 and code[i - 1] == ("s_nop", "0") and code[i - 2][0] == "s_add_u32" and code[i - 2][1].startswith("m0,")
            if not own:
                bad.append((i, "a transfer without its own M0", op, rest))
        elif re.search(r"\bm0\b", rest):
            if not (op == "s_add_u32" and rest.startswith("m0,") and not re.search(r"\bm0\b", rest[3:]) and
                    i + 2 < len(code) and code[i + 1] == ("s_nop", "0") and code[i + 2][0] and _is_transfer(*code[i + 2])):
                bad.append((i, "M0 used by something else", op, rest))
    # ages, in wait states, of vector-ALU writes on any path
    seen, todo = {}, [(0, {})]
    while todo:
        i, ages = todo.pop()
        old = seen.get(i)
        if old is not None:
            merged = dict(old)
            for r, a in ages.items():
                merged[r] = min(a, merged.get(r, SGPR_STATES))
            if merged == old:
                continue
            ages = merged
        seen[i] = ages
        op, rest = code[i]
        if op is not None:
            if op.startswith("v_mfma"):
                reads = _registers(rest.partition(",")[2])
                if any(kind == "v" and ages.get((kind, n), VGPR_STATES) < VGPR_STATES for kind, n in reads):
                    bad.append((i, "an operand written right before", op, rest))
            elif _is_transfer(op, rest):
                if any(kind == "s" and (kind, n) in ages for kind, n in _registers(rest)):
                    bad.append((i, "a scalar written right before", op, rest))
            wait = int(rest, 0) + 1 if op == "s_nop" else 1
            ages = {r: a + wait for r, a in ages.items() if a + wait < SGPR_STATES}
            ages.update({r: 0 for r in _vector_writes(op, rest)})
        todo += [(j, ages) for j in _successors(code, labels, i)]
    return products, transfers, sorted(set(bad))


@pytest.mark.skipif(not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")), reason="needs hipcc")
@pytest.mark.parametrize("extra", [[], ["-DAWQ_LDS_POISON"]], ids=["library", "lds_poison"])
def test_what_the_assembly_relies_on(tmp_path, extra):
    out = str(tmp_path / "gemm.s")
    subprocess.run([build.hipcc(), *build.FLAGS, *extra, "--cuda-device-only", "-S",
                    os.path.join(build.CSRC, "awq_mx_gemm.hip"), "-o", out], check=True, capture_output=True)
    with open(out) as f:
        kernels = _functions(f.read())
    assert len(kernels) == 12
    for name, code in kernels.items():
        products, transfers, bad = _check(code)
        assert products >= 64 and transfers >= 16 and not bad, (name, bad[:4])


MFMA = ("v_mfma_scale_f32_16x16x128_f8f6f4", "a[0:3], v[0:3], v[4:11], a[0:3], v12, v13 op_sel_hi:[0,0,0] cbsz:4")
M0, NOP, LOAD = ("s_add_u32", "m0, s9, 0x400"), ("s_nop", "0"), ("buffer_load_dwordx4", "v1, s[4:7], s8 offen lds")
END = ("s_endpgm", "")


def _offences(*code):
    return _check(list(code))[2]


def test_the_check_sees_mistakes():
    two = ("s_nop", "1")
    assert not _offences(MFMA, M0, NOP, LOAD, END)
    # M0
    assert _offences(LOAD, END) and _offences(M0, LOAD, END) and _offences(M0, NOP, LOAD, LOAD, END)
    assert _offences(("s_mov_b32", "m0, s1"), M0, NOP, LOAD, END)
    assert _offences(("s_add_u32", "m0, m0, 0x400"), NOP, LOAD, END)
    assert _offences(M0, NOP, ("s_add_u32", "s1, m0, 4"), END)
    # elements and scales
    for reg in ("v2", "v7", "v12", "v13"):
        write = ("v_mov_b32_e32", f"{reg}, v40")
        assert _offences(write, MFMA, END) and _offences(write, NOP, MFMA, END) and not _offences(write, two, MFMA, END)
    assert _offences(("v_permlane16_swap_b32", "v40, v5"), MFMA, END)
    assert not _offences(("v_mov_b32_e32", "v40, v2"), MFMA, END)
    loop = [(None, ".L1"), MFMA, ("v_lshlrev_b32_e32", "v3, 1, v40"), ("s_cbranch_scc1", ".L1"), END]
    assert _offences(*loop) and not _offences(*loop[:3], two, *loop[3:])
    # scalars
    for reg in ("s4", "s7", "s8"):
        write = ("v_readfirstlane_b32", f"{reg}, v40")
        assert _offences(write, M0, NOP, LOAD, END) and not _offences(write, ("s_nop", "2"), M0, NOP, LOAD, END)
    assert _offences(("v_cmp_eq_u32_e64", "s[8:9], v1, v2"), M0, NOP, LOAD, END)
    assert not _offences(("s_mov_b32", "s8, 0"), M0, NOP, LOAD, END)
