"""The 8-bit linear-layer operators on the GPU against plain references in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

from tests import linear_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def fp4q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import fp4_communication_compression_amd as m
    m.lib()
    return m


def rand(gen, rows, cols, dtype, scale=1.0):
    v = torch.randn(rows, cols, generator=gen) * torch.exp(torch.randn(rows, 1, generator=gen))
    return (v * scale).to(dtype)


def up(t):
    """To the GPU; 8-bit codes with the padded rows that they have here."""
    if t is None or t.element_size() > 1:
        return None if t is None else t.to(DEV)
    rows, pitch = t.shape[0], (t.shape[1] + 15) // 16 * 16
    room = torch.as_strided(t.view(torch.uint8), (rows, pitch), (pitch, 1)).to(DEV)
    return room.view(t.dtype)[:, :t.shape[1]]


def down(t):
    return t.cpu() if t.element_size() > 1 else t.contiguous().view(torch.uint8).cpu().view(t.dtype)


def within(got, want, off):
    bad = (got.double() - want).abs() > off
    assert not bool(bad.any()), "%d of %d out of bounds, worst %.3g of the bound" % (
        int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / off.clamp_min(1e-300)).max()))


def same(a, b):
    """Equal values, NaN where NaN."""
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


# ------------------------------------------------------------------ quantise
QUANT_SHAPES = [(1, 1), (1, 128), (3, 130), (17, 64), (128, 128), (129, 127), (200, 1000), (130, 5003),
                (257, 384), (8, 4096)]


def check_codes(codes, scales, v, fmt, tiles):
    want, want_scales = ref.quantize(v, fmt, tiles)
    assert same(scales.cpu(), want_scales)
    assert same(down(codes).float(), want)   # as values: zeros have no sign


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", QUANT_SHAPES)
@pytest.mark.parametrize("tiles", [False, True])
def test_quantize_matches_the_definition_exactly(fp4q, shape, dtype, fmt, tiles):
    x = rand(torch.Generator().manual_seed(sum(shape)), *shape, dtype)
    q = fp4q.fp4q_quantize8(x.to(DEV), fmt, tiles=tiles, transposed=True)
    check_codes(q.codes, q.scales, x.float(), fmt, tiles)
    check_codes(q.codes_t, q.scales_t, x.float().t().contiguous(), fmt, tiles)
    one = fp4q.fp4q_quantize8(x.to(DEV), fmt, tiles=tiles)
    other = fp4q.fp4q_quantize8(x.to(DEV), fmt, tiles=tiles, straight=False, transposed=True)
    assert one.codes_t is None and other.codes is None
    assert torch.equal(down(one.codes).float(), down(q.codes).float()) and torch.equal(one.scales, q.scales)
    assert torch.equal(down(other.codes_t).float(), down(q.codes_t).float())
    assert torch.equal(other.scales_t, q.scales_t)


def test_quantize_rows_of_no_height(fp4q):
    q = fp4q.fp4q_quantize8(torch.empty(0, 300, dtype=BF16, device=DEV), transposed=True)
    assert q.codes.shape == (0, 300) and q.scales.shape == (3, 0)
    assert q.codes_t.shape == (300, 0) and q.scales_t.shape == (0, 300)


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("tiles", [False, True])
def test_quantize_edges(fp4q, fmt, tiles):
    """Blocks of zeros, of values near fp32's ends, of format borders, not finite."""
    x = torch.zeros(256, 640)
    x[:, 128:256] = torch.randn(256, 128, generator=torch.Generator().manual_seed(1)) * 2.0 ** -90
    x[:, 256:384] = torch.linspace(-3.3e38, 3.3e38, 128)
    x[:, 384:512] = torch.arange(128) * 2.0 ** -9
    x[:, 512:] = torch.linspace(-1, 1, 128) * 3.4e38
    q = fp4q.fp4q_quantize8(x.to(DEV), fmt, tiles=tiles, transposed=True)
    check_codes(q.codes, q.scales, x, fmt, tiles)
    check_codes(q.codes_t, q.scales_t, x.t().contiguous(), fmt, tiles)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quantize_marks_blocks_that_are_not_finite(fp4q, bad):
    x = torch.ones(130, 300)
    x[129, 140] = bad
    q = fp4q.fp4q_quantize8(x.to(DEV), transposed=True)
    codes, scales = down(q.codes).float(), q.scales.cpu()
    assert bool(codes[129, 128:256].isnan().all()) and bool(scales[1, 129].isnan())
    assert int(codes.isnan().sum()) == 128 and int(scales.isnan().sum()) == 1
    codes, scales = down(q.codes_t).float(), q.scales_t.cpu()
    assert bool(codes[140, 128:].isnan().all()) and int(codes.isnan().sum()) == 2
    assert bool(scales[1, 140].isnan()) and int(scales.isnan().sum()) == 1
    q = fp4q.fp4q_quantize8(x.to(DEV), tiles=True)
    assert int(down(q.codes).float().isnan().sum()) == 2 * 128 and int(q.scales.isnan().sum()) == 1


# ---------------------------------------------------------------------- norm
NORM_SHAPES = [(1, 1), (1, 4096), (2, 7), (5, 64), (33, 128), (4, 130), (9, 1000), (6, 1024), (7, 2048),
               (3, 4096), (3, 5003), (2, 8192), (5, 11008), (3, 16384), (2, 20000), (1, 65536), (2, 65544)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm(fp4q, shape, dtype, with_residual):
    gen = torch.Generator().manual_seed(shape[0] * 7 + shape[1])
    x, w = rand(gen, *shape, dtype), (1 + 0.2 * torch.randn(shape[1], generator=gen)).to(dtype)
    res = rand(gen, *shape, dtype) if with_residual else None
    out = fp4q.fp4q_rmsnorm(x.to(DEV), w.to(DEV), EPS, residual=up(res), want_codes=True, want_rstd=True)
    h = x if res is None else (x.float() + res.float()).to(dtype)
    assert torch.equal(out.h.cpu(), h)
    r, y = ref.norm(h, w, EPS)
    chain = max(ref.ROW_CHAIN, shape[1] // 256 + 22)
    # the squares' sum: its chain; then the mean, eps, root and reciprocal; the root halves
    # what came before it
    off_r = ((chain + 2) / 2 + 3) * ref.U
    within(out.rstd.cpu(), r, off_r * r)
    off_y = off_r + 2 * ref.U
    within(out.y.cpu(), y, (off_y + ref.HALF_STEP[dtype]) * y.abs())
    top = ref.blocks_amax(y, 1).t() / 448
    within(out.scales.cpu(), top, (off_y + 2 * ref.U) * top + 2.0 ** -100)
    wide = ref.spread(out.scales.cpu(), *shape)
    # half a step of a code: 2^-4 of a normal value, 2^-10 scales of a subnormal one
    within(ref.values(down(out.codes), out.scales.cpu()), y,
           (2.0 ** -4 + 2 * off_y) * y.abs() + (2.0 ** -10) * wide)
    for want_y, want_codes in ((True, False), (False, True)):
        part = fp4q.fp4q_rmsnorm(x.to(DEV), w.to(DEV), EPS, residual=up(res), want_y=want_y, want_codes=want_codes)
        assert part.rstd is None and (part.y is None) != want_y and (part.codes is None) != want_codes
        if want_y:
            assert torch.equal(part.y, out.y)
        else:
            assert torch.equal(down(part.codes).view(torch.uint8), down(out.codes).view(torch.uint8))
            assert torch.equal(part.scales, out.scales)


@pytest.mark.parametrize("cols", [256, 515])
def test_norm_updates_the_residual_in_place(fp4q, cols):
    gen = torch.Generator().manual_seed(3)
    x, res, w = (rand(gen, 37, cols, BF16).to(DEV) for _ in range(3))
    w = w[0].contiguous()
    want = fp4q.fp4q_rmsnorm(x, w, EPS, residual=res, want_codes=True)
    got = fp4q.fp4q_rmsnorm(x, w, EPS, residual=res, h=res, want_codes=True)
    assert got.h is res and torch.equal(want.h, res) and torch.equal(want.y, got.y)
    assert torch.equal(want.scales, got.scales)


def test_norm_edges(fp4q):
    """A row of zeros, a NaN, an infinity, values whose squares leave bf16's range."""
    x = torch.ones(6, 256, dtype=F32)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    x[3] = 1e-18
    x[4] = 1e17
    w = torch.ones(256)
    out = fp4q.fp4q_rmsnorm(x.to(DEV), w.to(DEV), EPS, want_codes=True, want_rstd=True)
    y, scales, codes = out.y.cpu(), out.scales.cpu(), down(out.codes).float()
    assert bool((y[0] == 0).all()) and bool((codes[0] == 0).all())
    assert bool(y[1].isnan().all()) and bool(codes[1].isnan().all()) and bool(scales[:, 1].isnan().all())
    assert bool(y[2, 200].isnan()) and bool(codes[2, 128:].isnan().all())   # inf * 0
    r, want = ref.norm(x, w, EPS)
    for i in (3, 4, 5):
        within(y[i], want[i], 60 * ref.U * want[i].abs())
    empty = fp4q.fp4q_rmsnorm(torch.empty(0, 256, device=DEV), w.to(DEV), EPS, want_codes=True)
    assert empty.y.shape == (0, 256) and empty.codes.shape == (0, 256)


# ------------------------------------------------------------ norm gradients
GRAD_SHAPES = [(1, 1), (1, 4096), (3, 7), (40, 64), (70, 130), (300, 1000), (33, 2048), (1500, 256), (65, 4096),
               (33, 5003), (9, 11008), (5, 16384), (3, 20000), (2, 65536), (2, 65544)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", GRAD_SHAPES)
@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_grad(fp4q, shape, dtype, with_dh):
    gen = torch.Generator().manual_seed(shape[0] * 5 + shape[1])
    h, w = rand(gen, *shape, dtype), (1 + 0.2 * torch.randn(shape[1], generator=gen)).to(dtype)
    dy, dh = rand(gen, *shape, dtype, 0.1), rand(gen, *shape, dtype, 0.1) if with_dh else None
    rstd = ref.norm(h, w, EPS)[0].float()
    dx, dw = fp4q.fp4q_rmsnorm_backward(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV), dh=up(dh))
    want, off, want_w, off_w = ref.norm_grad(dy, h, w, rstd, dh)
    if shape[1] // 256 + 22 > ref.ROW_CHAIN:
        off = off * (shape[1] // 256 + 22) / ref.ROW_CHAIN
    within(dx.cpu(), want, off + ref.HALF_STEP[dtype] * (want.abs() + off))
    within(dw.cpu(), want_w, off_w)


def test_norm_grad_against_differences(fp4q):
    """Directional derivatives of sum(y dy) + sum(h dh) in 64 bits, central differences."""
    gen = torch.Generator().manual_seed(11)
    h, w = torch.randn(4, 72, generator=gen), 1 + 0.2 * torch.randn(72, generator=gen)
    dy, dh = torch.randn(4, 72, generator=gen), torch.randn(4, 72, generator=gen)
    rstd = ref.norm(h, w, EPS)[0].float()
    dx, dw = (t.cpu().double() for t in fp4q.fp4q_rmsnorm_backward(
        dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV), dh=dh.to(DEV)))

    def loss(h, w):
        return float((ref.norm(h, w, EPS)[1] * dy.double()).sum() + (h * dh.double()).sum())

    step = 1e-4
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        vh, vw = torch.randn(4, 72, generator=g).double(), torch.randn(72, generator=g).double()
        hd, wd = h.double(), w.double()
        diff = (loss(hd + step * vh, wd + step * vw) - loss(hd - step * vh, wd - step * vw)) / (2 * step)
        size = float((dx * vh).abs().sum() + (dw * vw).abs().sum())
        # the differences' own error is about step^2 = 1e-8, the kernel's about 100 u
        assert abs(diff - float((dx * vh).sum() + (dw * vw).sum())) <= (200 * ref.U + 1e-6) * size


def test_norm_grad_of_no_rows(fp4q):
    e = torch.empty(0, 640, dtype=BF16, device=DEV)
    dx, dw = fp4q.fp4q_rmsnorm_backward(e, e, torch.ones(640, dtype=BF16, device=DEV),
                                        torch.empty(0, device=DEV))
    assert dx.shape == (0, 640) and bool((dw == 0).all())


# ------------------------------------------------------------------- product
GEMM_SHAPES = [(1, 1, 1), (1, 128, 128), (1, 257, 1000), (2, 5, 17), (7, 64, 127), (16, 130, 129), (17, 300, 4096),
               (33, 1000, 640), (48, 513, 2049), (64, 128, 256), (65, 129, 384), (100, 4096, 300),
               (128, 128, 1024), (129, 255, 15), (200, 384, 16), (256, 256, 512), (300, 520, 1111),
               (515, 777, 640), (1, 4096, 11008), (16, 256, 16400), (1030, 512, 128)]


def make(gen, m, n, k, fa, fb, tiles):
    a, b = ref.fake_codes(gen, m, k, fa), ref.fake_codes(gen, n, k, fb)
    g = ref.groups(k)
    sa = torch.rand(g, m, generator=gen) + 0.1
    sb = torch.rand(g, ref.groups(n) if tiles else n, generator=gen) + 0.1
    return a, sa, b, sb


def check_bf16(got, a, sa, b, sb):
    """Every value within its bound, and the whole within half a step of bf16 (dropped
    bits are far below that in the mean; one k of 16400 left out is 2^-7)."""
    want = ref.gemm(a, sa, b, sb)[0]
    within(got, want, ref.gemm_bf16_off(a, sa, b, sb, want))
    assert float((got.double() - want).norm()) <= ref.HALF_STEP[BF16] * float(want.norm())


@pytest.mark.parametrize("shape", GEMM_SHAPES)
@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("fa,fb", [(E4M3, E4M3), (E5M2, E4M3)])
def test_gemm(fp4q, shape, tiles, fa, fb):
    print("gemm", shape, tiles, fa, fb, flush=True)
    m, n, k = shape
    a, sa, b, sb = make(torch.Generator().manual_seed(m + n + k), m, n, k, fa, fb, tiles)
    want, off = ref.gemm(a, sa, b, sb)
    dev = [up(a), sa.to(DEV), up(b), sb.to(DEV)]
    got = fp4q.fp4q_gemm8(*dev, out_dtype=F32)
    within(got.cpu(), want, off)
    assert torch.equal(got, fp4q.fp4q_gemm8(*dev, out_dtype=F32))
    half = fp4q.fp4q_gemm8(*dev)
    assert half.dtype == BF16 and torch.equal(half, fp4q.fp4q_gemm8(*dev))
    check_bf16(half.cpu(), a, sa, b, sb)
    total = torch.randn(m, n, generator=torch.Generator().manual_seed(1))
    into = total.to(DEV)
    assert fp4q.fp4q_gemm8(*dev, out=into, accumulate=True) is into
    assert torch.equal(into, total.to(DEV) + got)


@pytest.mark.parametrize("fa", [E4M3, E5M2])
@pytest.mark.parametrize("fb", [E4M3, E5M2])
@pytest.mark.parametrize("m", [5, 140, 600])
def test_gemm_formats(fp4q, fa, fb, m):
    a, sa, b, sb = make(torch.Generator().manual_seed(m), m, 300, 450, fa, fb, True)
    want, off = ref.gemm(a, sa, b, sb)
    within(fp4q.fp4q_gemm8(up(a), sa.to(DEV), up(b), sb.to(DEV), out_dtype=F32).cpu(), want, off)
    check_bf16(fp4q.fp4q_gemm8(up(a), sa.to(DEV), up(b), sb.to(DEV)).cpu(), a, sa, b, sb)


@pytest.mark.parametrize("m,n", [(3, 70), (200, 300), (512, 512)])
def test_gemm_of_no_length(fp4q, m, n):
    a, b = torch.empty(m, 0, dtype=E4M3, device=DEV), torch.empty(n, 0, dtype=E4M3, device=DEV)
    s = torch.empty(0, m, device=DEV), torch.empty(0, n, device=DEV)
    assert bool((fp4q.fp4q_gemm8(a, s[0], b, s[1]) == 0).all())
    out = torch.ones(m, n, device=DEV)
    fp4q.fp4q_gemm8(a, s[0], b, s[1], out=out, accumulate=True)
    assert bool((out == 1).all())
    none = fp4q.fp4q_gemm8(torch.empty(0, 256, dtype=E4M3, device=DEV), torch.empty(2, 0, device=DEV),
                           torch.empty(n, 256, dtype=E4M3, device=DEV), torch.empty(2, n, device=DEV))
    assert none.shape == (0, n)


@pytest.mark.parametrize("m", [1, 20, 140, 300])
def test_gemm_of_slices(fp4q, m):
    """Operands that are column slices of wider tensors."""
    gen = torch.Generator().manual_seed(m)
    a, sa, b, sb = make(gen, m, 260, 1024, E4M3, E4M3, True)
    cut = slice(256, 256 + 400)
    want, off = ref.gemm(a[:, cut], sa[2:6], b[:, cut], sb[2:6])
    dev = a.to(DEV)[:, cut], sa[2:6].to(DEV), b.to(DEV)[:, cut], sb[2:6].to(DEV)
    within(fp4q.fp4q_gemm8(*dev, out_dtype=F32).cpu(), want, off)
    check_bf16(fp4q.fp4q_gemm8(*dev).cpu(), a[:, cut], sa[2:6], b[:, cut], sb[2:6])


@pytest.mark.parametrize("m", [1, 40, 300])
def test_gemm_carries_what_is_not_finite(fp4q, m):
    """A NaN scale or code reaches the outputs that it belongs to, and no others."""
    a, sa, b, sb = make(torch.Generator().manual_seed(m), m, 200, 300, E4M3, E4M3, False)
    sa[1, 0] = float("nan")
    b.view(torch.uint8)[77, 290] = 0x7F
    want = torch.zeros(m, 200, dtype=torch.bool)
    want[0] = True
    want[:, 77] = True
    for dtype in (BF16, F32):
        got = fp4q.fp4q_gemm8(up(a), sa.to(DEV), up(b), sb.to(DEV), out_dtype=dtype).cpu()
        assert torch.equal(got.isnan(), want)


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (300, 512, 4096), (600, 700, 900)])
def test_gemm_of_a_quantised_layer(fp4q, m, n, k):
    """Activations, weight and gradients through the quantiser, in the three directions: each
    product against its operands' own values."""
    gen = torch.Generator().manual_seed(5)
    x, w, dy = rand(gen, m, k, BF16), rand(gen, n, k, BF16, k ** -0.5), rand(gen, m, n, BF16)
    qx = fp4q.fp4q_quantize8(x.to(DEV), transposed=True)
    qw = fp4q.fp4q_quantize8(w.to(DEV), tiles=True, transposed=True)
    qd = fp4q.fp4q_quantize8(dy.to(DEV), E5M2, transposed=True)
    for a, sa, b, sb, shape in ((qx.codes, qx.scales, qw.codes, qw.scales, (m, n)),
                                (qd.codes, qd.scales, qw.codes_t, qw.scales_t, (m, k)),
                                (qd.codes_t, qd.scales_t, qx.codes_t, qx.scales_t, (n, k))):
        got = fp4q.fp4q_gemm8(a, sa, b, sb, out_dtype=F32)
        assert got.shape == shape
        want, off = ref.gemm(down(a), sa.cpu(), down(b), sb.cpu())
        within(got.cpu(), want, off)
        check_bf16(fp4q.fp4q_gemm8(a, sa, b, sb).cpu(), down(a), sa.cpu(), down(b), sb.cpu())


# ------------------------------------------------------- streams and graphs
def layer(fp4q, x, res, w, qw, stream=None):
    n = fp4q.fp4q_rmsnorm(x, w, EPS, residual=res, want_codes=True, want_rstd=True, stream=stream)
    out = fp4q.fp4q_gemm8(n.codes, n.scales, qw.codes, qw.scales, stream=stream)
    qd = fp4q.fp4q_quantize8(out, E5M2, transposed=True, stream=stream)
    dn = fp4q.fp4q_gemm8(qd.codes, qd.scales, qw.codes_t, qw.scales_t, stream=stream)
    qn = fp4q.fp4q_quantize8(n.y, straight=False, transposed=True, stream=stream)
    dw = fp4q.fp4q_gemm8(qd.codes_t, qd.scales_t, qn.codes_t, qn.scales_t, out_dtype=F32, stream=stream)
    dx, dg = fp4q.fp4q_rmsnorm_backward(dn, n.h, w, n.rstd, dh=x, stream=stream)
    return [out, dn, dw, dx, dg]


@pytest.mark.parametrize("rows", [3, 200])
def test_streams_and_graphs(fp4q, rows):
    """The same values on another stream and from a graph, replayed among eager work."""
    gen = torch.Generator().manual_seed(rows)
    x, res = rand(gen, rows, 520, BF16).to(DEV), rand(gen, rows, 520, BF16).to(DEV)
    w = torch.ones(520, dtype=BF16, device=DEV)
    qw = fp4q.fp4q_quantize8(rand(gen, 384, 520, BF16, 0.05).to(DEV), tiles=True, transposed=True)
    want = layer(fp4q, x, res, w, qw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer(fp4q, x, res, w, qw, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = layer(fp4q, x, res, w, qw)
    for turn in range(4):
        x.copy_(rand(gen, rows, 520, BF16).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        eager = layer(fp4q, x, res, w, qw)
        assert all(torch.equal(a, b) for a, b in zip(eager, held)), turn


# ------------------------------------------------- together, and past 32 bits
@pytest.mark.parametrize("ranks,tokens,hidden,inner", [(2, 96, 512, 1024), (4, 7, 256, 528), (1, 200, 512, 300)])
def test_example_layer(fp4q, ranks, tokens, hidden, inner):
    """The tensor-parallel layer of examples/tp_layer.py against fp32.  An 8-bit operand is off
    by at most 2^-4 (E4M3) or 2^-3 (E5M2) of a value, which random values average to at most
    0.04 and 0.08 of a product's norm; the layer chains two products with a square between
    (twice the first one's error) and as many back.  FP4 adds at most 0.25 a value, 0.15 in
    the norm, at each of two exchanges."""
    from examples import tp_layer
    plain = tp_layer.errors(ranks, tokens, hidden, inner, compress=False)
    fp4 = tp_layer.errors(ranks, tokens, hidden, inner, compress=True)
    print(plain, fp4, flush=True)
    assert max(plain.values()) < 0.2
    assert max(fp4.values()) < 0.5


def test_norm_past_32_bits(fp4q):
    rows, cols = 140000, 16384
    x = torch.zeros(rows, cols, dtype=BF16, device=DEV)
    tail = rand(torch.Generator().manual_seed(0), 5, cols, BF16)
    x[-5:] = tail.to(DEV)
    w = torch.ones(cols, dtype=BF16, device=DEV)
    out = fp4q.fp4q_rmsnorm(x, w, EPS, want_codes=True, want_rstd=True)
    r, y = ref.norm(tail, w.cpu(), EPS)
    within(out.y[-5:].cpu(), y, (60 * ref.U + 2.0 ** -8) * y.abs())
    within(ref.values(down(out.codes[-5:]), out.scales[:, -5:].cpu()), y, 2.0 ** -3.9 * y.abs() + 1e-2)
    assert bool((out.y[:3] == 0).all()) and bool((out.y[-9:-5] == 0).all())
    del out
    dy = torch.zeros_like(x)
    dy[-5:] = tail.flip(0).to(DEV)
    rstd = torch.zeros(rows, device=DEV)
    rstd[-5:] = r.float().to(DEV)
    dx, dw = fp4q.fp4q_rmsnorm_backward(dy, x, w, rstd)
    want, off, want_w, off_w = ref.norm_grad(tail.flip(0), tail, w.cpu(), r.float(), None)
    within(dx[-5:].cpu(), want, off + 2.0 ** -8 * (want.abs() + off))
    within(dw.cpu(), want_w, off_w)
    assert bool((dx[-9:-5] == 0).all())


def test_quantize_past_32_bits(fp4q):
    rows, cols = 140000, 16384
    x = torch.zeros(rows, cols, dtype=BF16, device=DEV)
    tail = rand(torch.Generator().manual_seed(0), 64, cols, BF16)   # rows 139936 ..: 32 of the last tile, 32 before
    x[-64:] = tail.to(DEV)
    q = fp4q.fp4q_quantize8(x, transposed=True)
    check_codes(q.codes[-64:], q.scales[:, -64:], tail.float(), E4M3, False)
    part = torch.zeros(cols, 256)                                   # rows 139776 .. 140032, two groups
    part[:, 160:224] = tail.float().t()
    want, scales = ref.quantize(part, E4M3, False)
    assert same(down(q.codes_t[:, 139776:]).float(), want[:, :224])
    assert same(q.scales_t[1092:].cpu(), scales)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gemm_past_32_bits(fp4q, dtype):
    m, n, k = 50000, 45000, 130
    gen = torch.Generator().manual_seed(0)
    a, sa, b, sb = make(gen, 300, 300, k, E4M3, E4M3, False)
    big_a = torch.zeros(m, 144, dtype=torch.uint8, device=DEV).view(E4M3)[:, :k]
    big_b = torch.zeros(n, 144, dtype=torch.uint8, device=DEV).view(E4M3)[:, :k]
    big_a.view(torch.uint8)[-300:] = a.view(torch.uint8).to(DEV)
    big_b.view(torch.uint8)[-300:] = b.view(torch.uint8).to(DEV)
    scale_a, scale_b = torch.ones(2, m, device=DEV), torch.ones(2, n, device=DEV)
    scale_a[:, -300:] = sa.to(DEV)
    scale_b[:, -300:] = sb.to(DEV)
    out = fp4q.fp4q_gemm8(big_a, scale_a, big_b, scale_b, out_dtype=dtype)
    got = out[-300:, -300:].cpu()
    if dtype == F32:
        within(got, *ref.gemm(a, sa, b, sb))
    else:
        check_bf16(got, a, sa, b, sb)
    assert bool((out[-301] == 0).all()) and bool((out[-300:, -301] == 0).all()) and bool((out[:2] == 0).all())


def test_gemm_of_a_long_sum(fp4q):
    """A contraction of 1.5 million: a tile's rows span 192 MB and more."""
    k = 1500000
    gen = torch.Generator().manual_seed(0)
    a, sa, b, sb = make(gen, 40, 300, k, E4M3, E4M3, True)
    va, vb = (ref.values(x, s).to(DEV) for x, s in ((a, sa), (b, sb)))
    want = (va @ vb.t()).cpu()
    off = (va.abs() @ vb.abs().t()).cpu() * ref.U * (2 * 128 + sa.shape[0] + 8)
    within(fp4q.fp4q_gemm8(up(a), sa.to(DEV), up(b), sb.to(DEV), out_dtype=F32).cpu(), want, off)
