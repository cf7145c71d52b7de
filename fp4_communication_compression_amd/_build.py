"""Builds libfp4q.so (gfx950 only) in place with hipcc."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", n)
           for n in ("fp4q_gemm8.hip", "fp4q_gated8.hip", "fp4q_gated_grad.hip", "fp4q.hip", "fp4q_norm.hip",
                     "fp4q_quant8.hip", "fp4q_gemv4.hip")]
HEADERS = [*(os.path.join(ROOT, "include", n) for n in ("fp4q.h", "fp4q_linear.h", "fp4q_gated.h")),
           *(os.path.join(HERE, "csrc", n) for n in ("fp4q_numerics.h", "fp4q_f8.h", "fp4q_act.h", "fp4q_gemm8_plan.h",
                                                     "fp4q_gemm8_tile.h", "fp4q_gated8_plan.h", "fp4q_gemv4_plan.h"))]
LIB = os.path.join(HERE, "libfp4q.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # the kernels reproduce an fp32 operation order: no contraction into FMA,
    # IEEE division, fp32 denormals kept
    "-ffp-contract=off",
    "-fno-gpu-flush-denormals-to-zero",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    # never emit packed fp32 arithmetic
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _run(cmd) -> str:
    """What the command says, but for one harmless warning; raises if it fails."""
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in (res.stdout + res.stderr).splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + " ".join(cmd) + "\n" + err)
    return err.strip()


def build(force: bool = True, verbose: bool = False) -> str:
    stale = not os.path.exists(LIB) or any(
        os.path.getmtime(s) > os.path.getmtime(LIB) for s in SOURCES + HEADERS)
    if not (force or stale):
        return LIB
    tmp = LIB + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as room:
        # one compiler process per source file, at most four at a time
        flags = [f for f in HIPCC_FLAGS if f != "-shared"]
        objects = [os.path.join(room, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(max_workers=4) as pool:
            said = list(pool.map(_run, [[HIPCC, *flags, "-c", s, "-o", o] for s, o in zip(SOURCES, objects)]))
        said.append(_run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objects, "-o", tmp]))
    if verbose and any(said):
        print("\n".join(filter(None, said)))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
