"""The gated operators' sources: the inline assembly that they share with the 8-bit product
declares the registers that it writes, and their host code runs clean under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only; the GPU code is not run)."""
import os
import re
import shlex
import subprocess

import pytest

from fp4_communication_compression_amd import _build

CSRC = os.path.join(_build.HERE, "csrc")
INCLUDE = os.path.join(_build.ROOT, "include")
NAMES = ["fp4q_gated8.hip", "fp4q_gated_grad.hip", "fp4q_gemv4.hip"]
needs_hipcc = pytest.mark.skipif(not os.path.exists(_build.HIPCC), reason="needs hipcc")


@needs_hipcc
@pytest.mark.parametrize("name", NAMES)
def test_assembly_that_writes_m0_says_so(name, tmp_path):
    out = str(tmp_path / "device.ll")
    res = subprocess.run([_build.HIPCC, "--offload-arch=gfx950", "-O0", "-std=c++17", "-I", INCLUDE,
                          "--offload-device-only", "-S", "-emit-llvm", "-Xclang", "-disable-llvm-passes",
                          os.path.join(CSRC, name), "-o", out], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    found = re.findall(r'\basm (?:sideeffect )?"([^"]*)", "([^"]*)"', open(out).read())
    writes = [(text, constraints) for text, constraints in found if re.search(r"\bs_\w+\s+m0\b", text)]
    assert bool(writes) == (name == "fp4q_gated8.hip")
    for text, constraints in writes:
        assert "~{m0}" in constraints.split(","), text


@needs_hipcc
def test_host_code_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "gated_driver")
    cmd = shlex.split(
        "%s --offload-arch=gfx950 -Wl,--unresolved-symbols=ignore-all --offload-host-only -O1 -g -std=c++17 "
        "-Xarch_host -fsanitize=address -Xarch_host -fsanitize=undefined "
        "-Xarch_host -fno-sanitize-recover=all -I %s %s %s -o %s" % (
            _build.HIPCC, INCLUDE, os.path.join(_build.ROOT, "tests", "sanitize", "gated_driver.cpp"),
            " ".join(os.path.join(CSRC, n) for n in NAMES), exe))
    built = subprocess.run(cmd, cwd=str(tmp_path), capture_output=True, text=True, timeout=600)
    assert built.returncode == 0, built.stdout + built.stderr
    ran = subprocess.run([exe], cwd=str(tmp_path), capture_output=True, text=True, timeout=120)
    assert ran.returncode == 0 and "gated driver ok" in ran.stdout, ran.stdout + ran.stderr
