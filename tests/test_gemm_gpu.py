"""The 8-bit product on the GPU where its arithmetic and its kernels can go wrong: every
kernel on several blocks of K, scales far from 1, products that cancel."""
import pytest

torch = pytest.importorskip("torch")

from tests import gemm_shapes
from tests import linear_ref as ref
from tests.test_linear_gpu import check_bf16, fp4q, up, within  # noqa: F401 (fp4q is the fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
BF16, F32 = torch.bfloat16, torch.float32

def codes(gen, rows, k, fmt):
    """Random codes on the GPU whose rows are padded to 16 bytes with NaN codes."""
    room = torch.full((rows, (k + 15) // 16 * 16), 0x7F, dtype=torch.uint8, device=DEV)
    room[:, :k] = torch.randn(rows, k, generator=gen, device=DEV).mul(8).to(fmt).view(torch.uint8)
    return room.view(fmt)[:, :k]


def operands(m, n, k, fa, fb, tiles):
    gen = torch.Generator(device=DEV).manual_seed(m + n + k)
    g = ref.groups(k)
    a, b = codes(gen, m, k, fa), codes(gen, n, k, fb)
    sa = torch.rand(g, m, generator=gen, device=DEV) + 0.1
    return a, sa, b, torch.rand(g, ref.groups(n) if tiles else n, generator=gen, device=DEV) + 0.1


# All of the output against 64 bits, computed on the GPU by plain float64 products.
@pytest.mark.parametrize("shape", gemm_shapes.F32)
@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("fa", [E4M3, E5M2])
@pytest.mark.parametrize("fb", [E4M3, E5M2])
def test_every_kernel_with_f32_output(fp4q, shape, tiles, fa, fb):
    print(shape, tiles, fa, fb, flush=True)
    m, n, k = shape[:3]
    assert gemm_shapes.plan(m, n, k, True) == shape[3:]
    ops = operands(m, n, k, fa, fb, tiles)
    got = fp4q.fp4q_gemm8(*ops, out_dtype=F32)
    within(got, *ref.gemm(*ops))
    assert torch.equal(got, fp4q.fp4q_gemm8(*ops, out_dtype=F32))
    total = torch.randn(m, n, device=DEV)
    into = total.clone()
    assert fp4q.fp4q_gemm8(*ops, out=into, accumulate=True) is into
    assert torch.equal(into, total + got)


@pytest.mark.parametrize("shape", gemm_shapes.BF16)
@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("fa", [E4M3, E5M2])
@pytest.mark.parametrize("fb", [E4M3, E5M2])
def test_every_kernel_with_bf16_output(fp4q, shape, tiles, fa, fb):
    print(shape, tiles, fa, fb, flush=True)
    m, n, k = shape[:3]
    assert gemm_shapes.plan(m, n, k, False) == shape[3:]
    ops = operands(m, n, k, fa, fb, tiles)
    got = fp4q.fp4q_gemm8(*ops)
    check_bf16(got, *ops)
    assert torch.equal(got, fp4q.fp4q_gemm8(*ops))


@pytest.mark.parametrize("f32,shape", [(f32, s) for f32, shapes in ((False, gemm_shapes.BF16), (True, gemm_shapes.F32))
                                       for s in shapes if s[3] > 32])
def test_every_kernel_carries_what_is_not_finite(fp4q, f32, shape):
    """A NaN scale and a NaN code in the last block of K reach their row and column, no others."""
    m, n, k = shape[:3]
    a, sa, b, sb = operands(m, n, k, E4M3, E4M3, False)
    sa[-1, 5] = float("nan")
    b.view(torch.uint8)[n - 3, k - 1] = 0x7F
    want = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    want[5] = True
    want[:, n - 3] = True
    got = fp4q.fp4q_gemm8(a, sa, b, sb, out_dtype=F32 if f32 else BF16)
    assert torch.equal(got.isnan(), want)


# every kernel of the product: few rows, and each size of tile
SIZES = [(5, 300), (40, 300), (1030, 4100), (2047, 4096), (4000, 4096)]


def scales(gen, k, rows, power):
    return (torch.rand(ref.groups(k), rows, generator=gen) + 1) * 2.0 ** power


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales_whose_product_overflows(fp4q, m, n, tiles, dtype):
    """Scales of 2^70 on both sides of a block whose sum is 0, and of 2^70 against 2^-70:
    every sum is finite.  (A block of zeros between large values has such a scale.)"""
    print(m, n, tiles, dtype, flush=True)
    gen, k = torch.Generator().manual_seed(m), 300
    a, b = ref.fake_codes(gen, m, k, E4M3), ref.fake_codes(gen, n, k, E4M3)
    a.view(torch.uint8)[::2, :128] = 0
    sa, sb = scales(gen, k, m, 0), scales(gen, k, ref.groups(n) if tiles else n, 0)
    sa[0, ::2] *= 2.0 ** 70
    sa[0, 1::2] *= 2.0 ** -70
    sb[0] *= 2.0 ** 70
    sa[2] *= 2.0 ** 90
    sb[2] *= 2.0 ** -90
    got = fp4q.fp4q_gemm8(up(a), sa.to(DEV), up(b), sb.to(DEV), out_dtype=dtype).cpu()
    rows = torch.unique(torch.cat([torch.arange(0, m, 61), torch.arange(max(0, m - 9), m)]))
    part = a[rows], sa[:, rows], b, sb
    if dtype == F32:
        within(got[rows], *ref.gemm(*part))
    else:
        check_bf16(got[rows], *part)
    assert bool(got.isfinite().all())


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales_whose_product_underflows(fp4q, m, n, tiles, dtype):
    """Scales of 2^-73 on both sides under sums of 2^24: the results are normal numbers, the
    scales' product is not."""
    print(m, n, tiles, dtype, flush=True)
    gen, k = torch.Generator().manual_seed(m + 1), 300
    a, b = ref.fake_codes(gen, m, k, E5M2), ref.fake_codes(gen, n, k, E4M3)
    a.copy_((torch.randn(m, k, generator=gen) * 10000).to(E5M2))
    b.copy_((torch.randn(n, k, generator=gen) * 80).clamp(-448, 448).to(E4M3))
    sa, sb = scales(gen, k, m, -73), scales(gen, k, ref.groups(n) if tiles else n, -73)
    got = fp4q.fp4q_gemm8(up(a), sa.to(DEV), up(b), sb.to(DEV), out_dtype=dtype).cpu()
    rows = torch.unique(torch.cat([torch.arange(0, m, 61), torch.arange(max(0, m - 9), m)]))
    part = a[rows], sa[:, rows], b, sb
    want, off = ref.gemm(*part)
    if dtype == F32:
        # and where a step or the result lies below the normal numbers, half of 2^-149 each
        within(got[rows], want, off + 8 * 2.0 ** -150)
    else:
        within(got[rows], want, ref.gemm_bf16_off(*part, want) + 8 * 2.0 ** -150 + 2.0 ** -134)


@pytest.mark.parametrize("m,n", [(5, 300), (40, 300), (2047, 4096), (4000, 4096)])
@pytest.mark.parametrize("fa", [E4M3, E5M2])
@pytest.mark.parametrize("tiles", [True, False])
def test_cancelling_products(fp4q, m, n, fa, tiles):
    """Of 8 neighbouring products two large ones cancel and the result is the sum of the small
    ones: bf16 output is off by at most 7 * 2^-13 of each group's largest product (and its own
    rounding), fp32 output by fp32's rounding alone."""
    print(m, n, fa, tiles, flush=True)
    k, gen = 256, torch.Generator().manual_seed(m)
    a, b = ref.fake_codes(gen, m, k, fa), ref.fake_codes(gen, n, k, E4M3)
    va, vb = torch.zeros(m, k), torch.zeros(n, k)
    for g in range(0, k, 8):
        at = (torch.randperm(8, generator=gen) + g).tolist()
        large = 2.0 ** torch.randint(4, 9, (m,), generator=gen)
        va[:, at[0]], va[:, at[1]] = large, -large
        vb[:, at[0]] = vb[:, at[1]] = 256
        for i in at[2:]:
            va[:, i] = 2.0 ** (6 * torch.rand(m, generator=gen) - 4)
            vb[:, i] = 2.0 ** (5 * torch.rand(n, generator=gen) - 2)
    a.copy_(va.to(fa))
    b.copy_(vb.to(E4M3))
    sa, sb = scales(gen, k, m, 0), scales(gen, k, ref.groups(n) if tiles else n, 0)
    rows = torch.unique(torch.cat([torch.arange(0, m, 193), torch.arange(max(0, m - 9), m)]))
    part = a[rows], sa[:, rows], b, sb
    want, off = ref.gemm(*part)
    dev = up(a), sa.to(DEV), up(b), sb.to(DEV)
    within(fp4q.fp4q_gemm8(*dev, out_dtype=F32).cpu()[rows], want, off)
    xa, xb = ref.values(*part[:2]), ref.values(*part[2:])
    for g in range(0, k, 8):
        top = torch.zeros_like(want)
        for i in range(g, g + 8):
            top = torch.maximum(top, (xa[:, i, None] * xb[None, :, i]).abs())
        off = off + 7 * 2.0 ** -13 * top
    half = ref.HALF_STEP[BF16]
    within(fp4q.fp4q_gemm8(*dev).cpu()[rows], want, off + half * (want.abs() + off))


def test_a_cancelled_sum_alone(fp4q):
    """448 * 448 - 448 * 448 + 2 * 2: fp32 output is exact, bf16 output within the bound."""
    a, b = torch.zeros(1, 128), torch.zeros(1, 128)
    a[0, :3] = torch.tensor([448.0, -448.0, 2.0])
    b[0, :3] = torch.tensor([448.0, 448.0, 2.0])
    one = torch.ones(1, 1, device=DEV)
    dev = a.to(E4M3).to(DEV), one, b.to(E4M3).to(DEV), one
    assert float(fp4q.fp4q_gemm8(*dev, out_dtype=F32)) == 4.0
    assert abs(float(fp4q.fp4q_gemm8(*dev)) - 4.0) <= 7 * 2.0 ** -13 * 448 * 448
