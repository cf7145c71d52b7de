"""The gated product of few rows: several units of 16 outputs a workgroup, and scales that are not
finite."""
import pytest

torch = pytest.importorskip("torch")

from tests import gated_shapes
from tests import linear_ref as ref
from tests.test_gated_gpu import E4M3, E5M2, check_gated, halves, operands
from tests.test_linear_gpu import fp4q  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu
STRIP = (64, 16, 1)


@pytest.mark.parametrize("shape", [(16, 4113, 1111), (7, 11008, 640), (1, 8209, 2300), (13, 4097, 4096), (2, 12290, 129)])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
def test_several_units_a_workgroup(fp4q, shape, fmt):
    """More units than the 256 workgroups: two or three each, the last ones fewer, whose sums take
    the two halves of their LDS in turn."""
    print(shape, fmt, flush=True)
    m, n, k = shape
    assert gated_shapes.plan(m, n, k) == STRIP and (n + 15) // 16 > 256
    ops = operands(m, n, k, fmt, fmt)
    got = fp4q.fp4q_gated8(*ops, "silu", want_pre=True)
    check_gated(got, halves(*ops), "silu", True)
    assert torch.equal(got.y, fp4q.fp4q_gated8(*ops, "silu").y)


@pytest.mark.parametrize("m,n,k", [(1, 33, 100), (5, 300, 300), (16, 4113, 640), (20, 300, 200), (40, 70, 1100), (300, 200, 300)])
def test_a_scale_that_is_infinite(fp4q, m, n, k):
    """An infinite scale of a's last block makes its row's products infinite, with the block's sign,
    in strips (whose wavefronts share K, some with a block less) as in tiles."""
    a, sa, w, sw = operands(m, n, k, seed=7)
    last = (k - 1) // 128 * 128
    codes, p = w.view(torch.uint8), ref.groups(n) * 128
    for half in (codes[:n, last:k], codes[p:, last:k]):
        half.copy_((half & 0x3F) | 1)         # positive, and not zero
    a.view(torch.uint8)[m - 1, last:k] = 0x38   # 1
    sa[-1, m - 1] = float("inf")
    got = fp4q.fp4q_gated8(a, sa, w, sw, "relu", want_pre=True)
    for t in (got.gate, got.up, got.y):
        assert bool((t[m - 1] == float("inf")).all()) and bool(t[:m - 1].isfinite().all())
