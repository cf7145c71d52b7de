"""The choice of kernel for a 4-bit product (host code, CPU only): the shapes that the GPU tests run
reach every kernel, with one unit of outputs a workgroup and with several, so that a change of the
choice cannot leave one untested."""
import itertools
import random

import pytest

from tests import gemv4_shapes as shapes
from tests.gemv4_shapes import BF16, F32, HELD, LOADED, STAGED, WIDE

KERNELS = [(STAGED, 16), (STAGED, 8), (HELD, 16), (LOADED, 8), (WIDE, 8)]


def test_the_tested_products_reach_every_kernel():
    for m, n, k, bits, transformed, gated, *want in shapes.SHAPES:
        way, waves, _, _, units, _ = shapes.plan(m, n, k, bits, bits, transformed, gated)
        assert [way, waves, units] == want, (m, n, k, bits, transformed, gated, way, waves, units)
    for kernel, gated in itertools.product(KERNELS, (False, True)):
        here = [c for c in shapes.SHAPES if c[6:8] == kernel and c[5] == gated]
        # two units, which take the sums' two places once, and three or more, which come back to the first
        assert {min(c[8], 3) for c in here} >= {2, 3}, (kernel, gated)
        # (the gated kernel with x in registers is for more than one unit only)
        assert any(c[8] == 1 for c in here) or (kernel, gated) == ((HELD, 16), True)
        assert any(c[1] % 16 for c in here), (kernel, gated)    # a ragged last unit
        assert {c[3] for c in here} == {BF16, F32} or kernel == (STAGED, 8), (kernel, gated)


def test_every_choice_is_one_of_the_kernels():
    """Over the range of sizes: a chunk's rows and parts fit its column tiles, the wavefronts of a
    kernel that holds x have a block each, and LDS is the GPU's 160 KiB at most."""
    rng = random.Random(5)
    for _ in range(20000):
        m, n, k = (int(2 ** rng.uniform(0, top)) for top in (12, 20, 10))
        k = 256 * min(k, 65535)
        bits, out, transformed, gated = rng.choice([BF16, F32]), rng.choice([BF16, F32]), rng.random() < 0.5, rng.random() < 0.5
        way, waves, each, chunks, units, lds = shapes.plan(m, n, k, bits, out, transformed, gated)
        parts = 2 if bits == F32 or (transformed and out == F32) else 1
        assert (way, waves) in KERNELS
        assert each * parts == (32 if way == WIDE else 16) and chunks == -(-m // each)
        assert way == WIDE or chunks == 1
        assert way != HELD or k // 256 <= waves
        assert 0 < lds <= 160 * 1024 and units >= 1


@pytest.mark.parametrize("m,n,k,gated,way", [(1, 4096, 11008, False, STAGED), (1, 11008, 4096, True, STAGED),
                                             (16, 32768, 4096, False, HELD), (16, 11008, 4096, True, HELD),
                                             (16, 2752, 4096, True, LOADED), (64, 4096, 4096, False, WIDE)])
def test_products_of_a_layer(m, n, k, gated, way):
    assert shapes.plan(m, n, k, BF16, BF16, False, gated)[0] == way
