"""The choice of kernel for an 8-bit product (host code, CPU only): the shapes that the GPU
tests run reach every kernel, so that a change of the choice cannot leave one untested."""
import pytest

from tests import gemm_shapes as shapes


@pytest.mark.parametrize("f32", [False, True])
def test_the_tested_products_reach_every_kernel(f32):
    cases = shapes.F32 if f32 else shapes.BF16
    for m, n, k, *want in cases:
        assert list(shapes.plan(m, n, k, f32)) == want, (m, n, k)
    large = [(128, 128), (128, 256) if f32 else (256, 256)]
    for tile in [(16, 16), (32, 128), (64, 128)] + large:
        here = [c for c in cases if c[3:5] == tile]
        assert any(c[2] % 128 for c in here)                            # a ragged last block
        assert any(c[1] % (4 if f32 else 8) for c in here)              # and rows of the output
        assert any(c[1] % (4 if f32 else 8) == 0 for c in here)
        assert all(c[2] > 4 * 128 for c in here if tile != (16, 16))    # the steady state
        if tile != (16, 16):
            assert any(c[5] > 1 for c in here) and any(c[5] == 1 for c in here)


def test_few_rows_and_no_length():
    for f32 in (False, True):
        assert shapes.plan(1, 4096, 11008, f32) == (16, 16, 1)
        assert shapes.plan(16, 1, 1 << 22, f32) == (16, 16, 1)
        assert shapes.plan(17, 1, 0, f32)[2] == 1 and shapes.plan(4096, 4096, 0, f32)[2] == 1
