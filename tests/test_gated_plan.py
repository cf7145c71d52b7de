"""The choice of kernel for a gated 8-bit product (host code, CPU only): the shapes that the GPU
tests run reach every kernel, so that a change of the choice cannot leave one untested."""
import pytest

from tests import gated_shapes as shapes

TILES = [(64, 16), (32, 64), (64, 64), (128, 64), (192, 128), (256, 128)]


def test_the_tested_products_reach_every_kernel():
    for m, n, k, *want in shapes.SHAPES:
        assert list(shapes.plan(m, n, k)) == want, (m, n, k)
    for tile in TILES:
        here = [c for c in shapes.SHAPES if c[3:5] == tile]
        assert any(c[2] % 128 for c in here) and any(c[1] % 8 for c in here) and any(c[1] % 8 == 0 for c in here)
        assert all(c[2] > 4 * 128 for c in here)    # the steady state
        if tile == (64, 16):                        # one, two and up to four column tiles, two units a workgroup
            assert {min(c[0] // 16, 3) if c[0] % 16 == 0 else c[0] // 16 + 1 for c in here} >= {1, 2, 3}
            assert any(c[1] == 16 * 256 for c in here)
        else:
            assert any(c[5] > 1 for c in here) and any(c[5] == 1 for c in here)


@pytest.mark.parametrize("m,n,k,tile", [(1, 11008, 4096, (64, 16)), (16, 1 << 20, 1 << 22, (64, 16)),
                                        (2047, 2752, 4096, (192, 128)), (8192, 11008, 4096, (256, 128))])
def test_products_of_a_layer(m, n, k, tile):
    assert shapes.plan(m, n, k) == tile + (1,)


def test_no_length_takes_no_strip():
    """A strip loads a first block of K; the tiles load none where there is none."""
    for m in (1, 3, 16, 17, 64, 200, 4096):
        for n in (1, 70, 4096, 100000):
            tile_m, tile_n, parts = shapes.plan(m, n, 0)
            assert (tile_m, tile_n) in TILES[1:] and parts == 1
