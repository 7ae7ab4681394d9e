"""The 8-bit operators' host-side argument handling under AddressSanitizer and
UndefinedBehaviorSanitizer.

Every HIP source is compiled again with the sanitizers applied to its host half only (the "-Xarch_host"
form: device code is built as usual and never runs here), linked into a separate library in a temporary
directory, and driven by tests/fp8_host_checks.cpp.  Needs no GPU; a sanitizer report or a failed
expectation fails the test.
"""
import os
import shutil
import subprocess

import pytest

from weight_only_int4_act_amd import build

SAN = ["address", "undefined"]
HERE = os.path.dirname(os.path.abspath(__file__))


def _tool(name):
    for p in (shutil.which(name), f"/opt/rocm/bin/{name}", f"/opt/rocm/llvm/bin/{name}"):
        if p and os.path.exists(p):
            return p
    pytest.skip(f"{name} not found")


@pytest.mark.slow
def test_8_bit_argument_checks_under_sanitizers(tmp_path):
    hipcc, clang = _tool("hipcc"), _tool("clang++")
    host = []
    for s in SAN:
        host += ["-Xarch_host", f"-fsanitize={s}"]
    host += ["-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-Wno-unused-command-line-argument"]
    objs = [str(tmp_path / (src + ".o")) for src in build.SOURCES]
    procs = [subprocess.Popen([hipcc, *flags, *host, "-c", os.path.join(build.CSRC, src), "-o", obj],
                              stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
             for src, obj in zip(build.SOURCES, objs)]
    for p, src in zip(procs, build.SOURCES):
        _, err = p.communicate()
        assert p.returncode == 0, f"{src}:\n{err[-4000:]}"
    lib, exe = str(tmp_path / "libawq_san.so"), str(tmp_path / "fp8_host_checks")
    link = [hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", lib]
    san = ",".join(SAN)
    main = [clang, "-std=c++17", "-O1", "-g", f"-fsanitize={san}", "-fno-sanitize-recover=undefined",
            "-fno-omit-frame-pointer", os.path.join(HERE, "fp8_host_checks.cpp"), lib, f"-Wl,-rpath,{tmp_path}", "-o", exe]
    for cmd in (link, main):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stderr[-4000:]}"
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "0 failures" in r.stdout, f"{r.stdout[-4000:]}\n{r.stderr[-6000:]}"
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-6000:]
