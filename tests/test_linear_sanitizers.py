"""The host code of the 8-bit linear-layer operators under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only; the GPU code is not built):
tests/sanitize/linear_driver.cpp calls every entry point with arguments that its validation
rejects, over sizes up to the ends of their types."""
import os
import shlex
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_host_code_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "linear_driver")
    csrc = os.path.join(ROOT, "fp4_communication_compression_amd", "csrc")
    cmd = shlex.split(
        "%s --offload-arch=gfx950 -Wl,--unresolved-symbols=ignore-all --offload-host-only -O1 -g -std=c++17 "
        "-Xarch_host -fsanitize=address -Xarch_host -fsanitize=undefined "
        "-Xarch_host -fno-sanitize-recover=all -I %s %s %s -o %s" % (
            HIPCC, os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "sanitize", "linear_driver.cpp"),
            " ".join(os.path.join(csrc, n) for n in ("fp4q_norm.hip", "fp4q_quant8.hip", "fp4q_gemm8.hip")), exe))
    built = subprocess.run(cmd, cwd=str(tmp_path), capture_output=True, text=True, timeout=600)
    assert built.returncode == 0, built.stdout + built.stderr
    ran = subprocess.run([exe], cwd=str(tmp_path), capture_output=True, text=True, timeout=120)
    assert ran.returncode == 0 and "linear driver ok" in ran.stdout, ran.stdout + ran.stderr
