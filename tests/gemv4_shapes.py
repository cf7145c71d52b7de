"""4-bit products that between them run every kernel of fp4q_gemv4 and fp4q_gated4, with one unit of
outputs a workgroup and with several: (M, N, K, bits of x, transformed, gated, way, wavefronts, units
a workgroup takes at most).  tests/test_gemv4_plan.py checks that they still do."""
import ctypes
import functools
import importlib.util
import os

HERE = os.path.dirname(os.path.abspath(__file__))
STAGED, HELD, LOADED, WIDE = range(4)
BF16, F32 = 16, 32

SHAPES = [
    # x made ready by the workgroups, 16 wavefronts and 8
    (1, 300, 11008, BF16, False, False, STAGED, 16, 1), (8, 4099, 4096, BF16, False, False, STAGED, 16, 2),
    (2, 12291, 4352, F32, False, False, STAGED, 16, 4), (4, 8209, 2304, BF16, True, False, STAGED, 16, 3),
    (3, 700, 1024, BF16, False, False, STAGED, 8, 1), (1, 8209, 2048, F32, True, False, STAGED, 8, 2),
    (5, 16401, 1280, BF16, False, False, STAGED, 8, 3),
    (8, 300, 2304, BF16, False, True, STAGED, 16, 1), (4, 4113, 2304, F32, True, True, STAGED, 16, 2),
    (5, 8195, 2048, BF16, False, True, STAGED, 16, 3),
    (1, 11008, 4096, BF16, False, True, STAGED, 8, 2), (2, 333, 4096, F32, False, True, STAGED, 8, 1),
    (3, 16387, 768, BF16, True, True, STAGED, 8, 3),
    # x in registers for all units
    (16, 4099, 4096, BF16, False, False, HELD, 16, 2), (16, 8209, 3840, BF16, False, False, HELD, 16, 3),
    (5, 5003, 4096, F32, True, False, HELD, 16, 2), (8, 12305, 2816, F32, True, False, HELD, 16, 4),
    (16, 130, 4096, BF16, False, False, HELD, 16, 1),
    (16, 4113, 4096, BF16, False, True, HELD, 16, 2), (16, 11008, 4096, BF16, True, True, HELD, 16, 3),
    (7, 4100, 3328, F32, True, True, HELD, 16, 2), (8, 8195, 4096, F32, False, True, HELD, 16, 3),
    # x loaded with each block
    (16, 130, 4352, BF16, False, False, LOADED, 8, 1), (16, 4113, 4352, BF16, False, False, LOADED, 8, 2),
    (6, 8195, 4608, F32, True, False, LOADED, 8, 3),
    (16, 2752, 4096, BF16, True, True, LOADED, 8, 1), (16, 4113, 4352, BF16, False, True, LOADED, 8, 2),
    (7, 8200, 4608, F32, True, True, LOADED, 8, 3),
    # two column tiles, whole chunks of rows and a last one of few
    (17, 333, 512, BF16, False, False, WIDE, 8, 1), (33, 8225, 512, BF16, False, False, WIDE, 8, 2),
    (9, 16417, 768, F32, True, False, WIDE, 8, 3),
    (40, 300, 1024, BF16, True, True, WIDE, 8, 1), (33, 4113, 512, F32, False, True, WIDE, 8, 2),
    (64, 8209, 256, BF16, False, True, WIDE, 8, 3),
]


@functools.lru_cache(None)
def _library():
    path = os.path.join(HERE, "hip", "libfp4q_gemv4_plan.so")
    if not os.path.exists(path):
        spec = importlib.util.spec_from_file_location("hip_build", os.path.join(HERE, "hip", "build.py"))
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        mod.build()
    return ctypes.CDLL(path)


def plan(m, n, k, x_bits, out_bits, transformed, gated):
    """What the library's own rule gives a product: the way, wavefronts, rows of x a chunk holds,
    chunks, units a workgroup takes at most, bytes of LDS."""
    out = (ctypes.c_int64 * 6)()
    _library().fp4q_gemv4_plan(ctypes.c_int64(m), ctypes.c_int64(n), ctypes.c_int64(k), int(x_bits == F32),
                               int(out_bits == F32), int(transformed), int(gated), out)
    return tuple(out)
