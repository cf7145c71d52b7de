"""Gated products that between them run every kernel of fp4q_gated8, whole and in runs of K, with
whole and ragged rows of the output: (M, N, K, rows of the kernel's tile, its outputs, runs of
K).  tests/test_gated_plan.py checks that they still do."""
import ctypes
import functools
import importlib.util
import os

HERE = os.path.dirname(os.path.abspath(__file__))

SHAPES = [(16, 2048, 1111, 64, 16, 1), (3, 133, 2222, 64, 16, 1), (24, 260, 900, 64, 16, 1), (64, 333, 2222, 64, 16, 1),
          (32, 4096, 1111, 64, 16, 1), (40, 4096, 1000, 64, 16, 1),
          (600, 260, 900, 32, 64, 1), (4296, 40, 1277, 32, 64, 1), (100, 257, 2222, 32, 64, 6), (48, 264, 4222, 32, 64, 7),
          (5000, 260, 1111, 64, 64, 1), (2049, 752, 640, 64, 64, 1), (37, 8486, 2266, 64, 64, 3),
          (1030, 3000, 1111, 128, 64, 1), (4099, 750, 1024, 128, 64, 1), (6000, 129, 4001, 128, 64, 3),
          (2047, 2752, 1000, 192, 128, 1), (2000, 2745, 1111, 192, 128, 1), (130, 4100, 16000, 192, 128, 7),
          (2049, 3000, 1111, 256, 128, 1), (3000, 2050, 1024, 256, 128, 1), (17717, 72, 7568, 256, 128, 3)]


@functools.lru_cache(None)
def _library():
    path = os.path.join(HERE, "hip", "libfp4q_gated8_plan.so")
    if not os.path.exists(path):
        spec = importlib.util.spec_from_file_location("hip_build", os.path.join(HERE, "hip", "build.py"))
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        mod.build()
    return ctypes.CDLL(path)


def plan(m, n, k):
    """The tile and the runs that the library's own rule gives a gated product."""
    out = (ctypes.c_int * 3)()
    _library().fp4q_gated8_plan(ctypes.c_int64(m), ctypes.c_int64(n), ctypes.c_int64(k), out)
    return tuple(out)
