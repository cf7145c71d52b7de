"""Products that between them run every kernel of fp4q_gemm8 on several blocks of K, whole and
in runs, with whole and ragged rows of the output: (M, N, K, rows of the kernel's tile, its
columns, runs of K).  tests/test_gemm_plan.py checks that they still do."""
import ctypes
import functools
import importlib.util
import os

HERE = os.path.dirname(os.path.abspath(__file__))

BF16 = [(16, 4096, 1111, 16, 16, 1), (3, 257, 2222, 16, 16, 1),
        (600, 520, 900, 32, 128, 1), (48, 513, 2222, 32, 128, 6),
        (5000, 520, 1111, 64, 128, 1), (2049, 1500, 640, 64, 128, 1), (3000, 257, 2222, 64, 128, 3),
        (1030, 6000, 1111, 128, 128, 1), (4099, 1500, 1024, 128, 128, 1), (6000, 257, 4001, 128, 128, 3),
        (2049, 6000, 1111, 256, 256, 1), (3000, 4100, 1024, 256, 256, 1), (130, 8200, 16000, 256, 256, 7)]
F32 = [(16, 4096, 1111, 16, 16, 1), (3, 257, 2222, 16, 16, 1),
       (600, 520, 900, 32, 128, 1), (48, 513, 2222, 32, 128, 6),
       (4000, 777, 1111, 64, 128, 1), (2049, 4096, 1024, 64, 128, 1), (1000, 257, 2222, 64, 128, 5),
       (4099, 1500, 1111, 128, 128, 1), (2049, 3001, 1024, 128, 128, 1), (6000, 257, 4001, 128, 128, 3),
       (1300, 4096, 6000, 128, 256, 1), (5000, 1030, 6016, 128, 256, 1), (1500, 2051, 9000, 128, 256, 2)]


@functools.lru_cache(None)
def _library():
    path = os.path.join(HERE, "hip", "libfp4q_gemm8_plan.so")
    if not os.path.exists(path):
        spec = importlib.util.spec_from_file_location("hip_build", os.path.join(HERE, "hip", "build.py"))
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        mod.build()
    return ctypes.CDLL(path)


def plan(m, n, k, f32):
    """The tile and the runs that the library's own rule gives a product."""
    out = (ctypes.c_int * 3)()
    _library().fp4q_gemm8_plan(ctypes.c_int64(m), ctypes.c_int64(n), ctypes.c_int64(k), int(f32), out)
    return tuple(out)
