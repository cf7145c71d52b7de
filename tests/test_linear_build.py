"""The 8-bit linear-layer kernels' inline assembly declares the registers that it writes, as
the compiler's own intermediate code of the device build shows it (CPU only)."""
import os
import re
import subprocess

import pytest

from fp4_communication_compression_amd import _build

CSRC = os.path.join(_build.HERE, "csrc")


@pytest.mark.skipif(not os.path.exists(_build.HIPCC), reason="needs hipcc")
@pytest.mark.parametrize("name", ["fp4q_norm.hip", "fp4q_quant8.hip", "fp4q_gemm8.hip"])
def test_assembly_that_writes_m0_says_so(name, tmp_path):
    out = str(tmp_path / "device.ll")
    res = subprocess.run([_build.HIPCC, "--offload-arch=gfx950", "-O0", "-std=c++17", "-I",
                          os.path.join(_build.ROOT, "include"), "--offload-device-only", "-S", "-emit-llvm", "-Xclang",
                          "-disable-llvm-passes", os.path.join(CSRC, name), "-o", out],
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    # call ... asm sideeffect "text", "constraints"
    found = re.findall(r'\basm (?:sideeffect )?"([^"]*)", "([^"]*)"', open(out).read())
    writes = [(text, constraints) for text, constraints in found if re.search(r"\bs_\w+\s+m0\b", text)]
    assert bool(writes) == (name == "fp4q_gemm8.hip")
    for text, constraints in writes:
        assert "~{m0}" in constraints.split(","), text
