"""The gated product's strips (host code, CPU only): only those of up to 16 rows give a workgroup more
than one unit of 16 outputs, and so need room in LDS for two units' sums."""
from tests import gated_shapes

STRIP = (64, 16, 1)


def test_units_of_a_workgroup():
    for m in (17, 24, 32, 33, 48, 64):
        for k in (1, 640, 4096, 4097, 11008):
            for n in (1, 16, 2752, 4095, 4096, 4097, 8192, 11008, 100000):
                assert gated_shapes.plan(m, n, k) != STRIP or -(-n // 16) <= 256, (m, n, k)
    assert all(gated_shapes.plan(m, 11008, 4096) == STRIP for m in range(1, 17))
