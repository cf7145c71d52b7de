"""The gated feed-forward operators on the GPU against plain references in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

from tests import gated_ref as gref
from tests import gated_shapes
from tests import linear_ref as ref
from tests.linear_ref import HALF_STEP, U
from tests.test_linear_gpu import down, fp4q, same, up, within  # noqa: F401 (fp4q is the fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
BF16, F32 = torch.bfloat16, torch.float32
ACTS = gref.ACTS


# ------------------------------------------------------------- 8-bit product
def codes(gen, rows, k, fmt, scale=8.0):
    """Random codes on the GPU whose rows are padded to 16 bytes with NaN codes."""
    room = torch.full((rows, (k + 15) // 16 * 16), 0x7F, dtype=torch.uint8, device=DEV)
    room[:, :k] = torch.randn(rows, k, generator=gen, device=DEV).mul(scale).to(fmt).view(torch.uint8)
    return room.view(fmt)[:, :k]


def joined(gen, n, k, fmt):
    """A joined weight whose padding rows hold NaN codes: nothing may come from them."""
    p = ref.groups(n) * 128
    w = codes(gen, p + n, k, fmt)
    w.view(torch.uint8)[n:p] = 0x7F
    return w


def operands(m, n, k, fa=E4M3, fw=E4M3, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(m + n + k + seed)
    g = ref.groups(k)
    a, w = codes(gen, m, k, fa), joined(gen, n, k, fw)
    sa = (torch.rand(g, m, generator=gen, device=DEV) + 0.1) * (0.02 * k ** -0.5)
    return a, sa, w, torch.rand(g, 2 * ref.groups(n), generator=gen, device=DEV) + 0.1


def halves(a, sa, w, sw):
    """Both products in 64 bits and the bounds of the 8-bit matrix core's fp32 sums."""
    n = w.shape[0] - sw.shape[1] // 2 * 128
    p, t = w.shape[0] - n, sw.shape[1] // 2
    va = ref.values(a, sa)
    out = []
    for rows, scales in ((w[:n], sw[:, :t]), (w[p:], sw[:, t:])):
        vw = ref.values(rows, scales)
        want = va @ vw.t()
        out.append((want, (va.abs() @ vw.abs().t()) * (7 * 2.0 ** -13 + U * (2 * 128 + sa.shape[0] + 8))))
    return out


def check_gated(got, want, act, pre):
    (g, off_g), (u, off_u) = want
    half = HALF_STEP[BF16]
    if pre:
        for t, w, off in ((got.gate, g, off_g), (got.up, u, off_u)):
            within(t, w, off + half * (w.abs() + off))
            assert float((t.double() - w).norm()) <= half * float(w.norm())
    else:
        assert got.gate is None and got.up is None
    value, slope, off, _ = gref.activate(g, act)
    # the derivative is at most 1.2, its change at most 1 for a change of 1 in g
    off = off + off_g * (1.2 + off_g)
    y, off_y = value * u, off * (u.abs() + off_u) + value.abs() * off_u
    within(got.y, y, off_y + half * (y.abs() + off_y) + 2 * U * y.abs())
    assert float((got.y.double() - y).norm()) <= half * float(y.norm()) + 2.0 ** -100


SMALL = [(1, 1, 1), (1, 128, 128), (1, 257, 1000), (2, 5, 17), (7, 64, 127), (16, 130, 129), (16, 8, 4096), (17, 300, 640),
         (33, 100, 640), (48, 257, 2049), (64, 64, 256), (65, 129, 384), (129, 127, 15), (200, 192, 16), (515, 388, 640),
         (1, 1376, 4096), (3, 2752, 4096)]


@pytest.mark.parametrize("shape", SMALL)
@pytest.mark.parametrize("act", ACTS)
def test_gated(fp4q, shape, act):
    print(shape, act, flush=True)
    ops = operands(*shape)
    want = halves(*ops)
    got = fp4q.fp4q_gated8(*ops, act, want_pre=True)
    assert got.y.dtype == got.gate.dtype == got.up.dtype == BF16 and got.y.shape == shape[:2]
    check_gated(got, want, act, True)
    alone = fp4q.fp4q_gated8(*ops, act)
    check_gated(alone, want, act, False)
    assert torch.equal(alone.y, got.y)


@pytest.mark.parametrize("shape", gated_shapes.SHAPES)
@pytest.mark.parametrize("fa", [E4M3, E5M2])
@pytest.mark.parametrize("fw", [E4M3, E5M2])
def test_every_kernel(fp4q, shape, fa, fw):
    print(shape, fa, fw, flush=True)
    m, n, k = shape[:3]
    assert gated_shapes.plan(m, n, k) == shape[3:]
    ops = operands(m, n, k, fa, fw)
    got = fp4q.fp4q_gated8(*ops, "silu", want_pre=True)
    check_gated(got, halves(*ops), "silu", True)
    assert torch.equal(got.y, fp4q.fp4q_gated8(*ops, "silu").y)


@pytest.mark.parametrize("m,n", [(5, 300), (40, 300), (1030, 2050), (2047, 2048), (4000, 2048)])
def test_scales_whose_product_leaves_the_range(fp4q, m, n):
    """Scales of 2^70 on both sides of a block whose sum is 0, and of 2^70 against 2^-70 and the
    gate's against the up projection's: every sum is finite."""
    print(m, n, flush=True)
    k = 300
    a, sa, w, sw = operands(m, n, k, seed=3)
    a.view(torch.uint8)[::2, :128] = 0
    t = sw.shape[1] // 2
    sa[0, ::2] *= 2.0 ** 70
    sa[0, 1::2] *= 2.0 ** -70
    sw[0, :t] *= 2.0 ** 70
    sw[0, t:] *= 2.0 ** 69
    sa[2] *= 2.0 ** 90
    sw[2] *= 2.0 ** -90
    got = fp4q.fp4q_gated8(a, sa, w, sw, "silu", want_pre=True)
    check_gated(got, halves(a, sa, w, sw), "silu", True)
    assert bool(got.y.isfinite().all())


@pytest.mark.parametrize("m", [1, 40, 300, 2100])
def test_gated_carries_what_is_not_finite(fp4q, m):
    """A NaN scale or code reaches the outputs that it belongs to, and no others."""
    n, k = 1200, 300
    a, sa, w, sw = operands(m, n, k, seed=5)
    sa[-1, 0] = float("nan")
    p = w.shape[0] - n
    w.view(torch.uint8)[p + 77, k - 1] = 0x7F   # a row of the up projection
    w.view(torch.uint8)[99, 3] = 0x7F           # and one of the gate
    got = fp4q.fp4q_gated8(a, sa, w, sw, "relu", want_pre=True)
    nan = [torch.zeros(m, n, dtype=torch.bool, device=DEV) for _ in range(2)]
    nan[0][0], nan[1][0], nan[0][:, 99], nan[1][:, 77] = True, True, True, True
    assert torch.equal(got.gate.isnan(), nan[0]) and torch.equal(got.up.isnan(), nan[1])
    assert torch.equal(got.y.isnan(), nan[0] | nan[1])


@pytest.mark.parametrize("m,n", [(3, 70), (200, 300), (2048, 1100)])
def test_gated_of_no_length(fp4q, m, n):
    r = ref.groups(n) * 128 + n
    a, w = torch.empty(m, 0, dtype=E4M3, device=DEV), torch.empty(r, 0, dtype=E4M3, device=DEV)
    s = torch.empty(0, m, device=DEV), torch.empty(0, ref.groups(r), device=DEV)
    got = fp4q.fp4q_gated8(a, s[0], w, s[1], want_pre=True)
    assert all(t.shape == (m, n) and bool((t == 0).all()) for t in got)
    none = fp4q.fp4q_gated8(torch.empty(0, 256, dtype=E4M3, device=DEV), torch.empty(2, 0, device=DEV),
                            torch.zeros(r, 256, dtype=torch.uint8, device=DEV).view(E4M3),
                            torch.ones(2, ref.groups(r), device=DEV), want_pre=True)
    assert none.y.shape == none.up.shape == (0, n)


@pytest.mark.parametrize("m", [2, 40])
def test_gated_past_32_bits(fp4q, m):
    """A joined weight of more than 4 GiB: its last columns against the product of them alone."""
    n, k, tail = 600000, 4096, 256
    gen = torch.Generator(device=DEV).manual_seed(1)
    p = ref.groups(n) * 128
    w = torch.zeros(p + n, k, dtype=torch.uint8, device=DEV)
    a, sa, part, sp = operands(m, tail, k)
    first = n - tail            # 599744 is not a multiple of 128: give all tiles one scale
    w[first:n] = part.view(torch.uint8)[:tail]
    w[p + first:] = part.view(torch.uint8)[tail:]
    sw = torch.full((k // 128, 2 * ref.groups(n)), 0.25, device=DEV)
    got = fp4q.fp4q_gated8(a, sa, w.view(E4M3), sw, "relu", want_pre=True)
    check_gated(fp4q.Gated8(*(t[:, first:] for t in got)), halves(a, sa, part, torch.full_like(sp, 0.25)), "relu", True)
    assert bool((got.gate[:, :first] == 0).all()) and bool((got.up[:, :first] == 0).all())


# ----------------------------------------------------------------- gradients
GRAD_SHAPES = [(1, 1), (1, 128), (3, 130), (17, 64), (128, 128), (129, 127), (200, 1000), (130, 2503), (257, 384), (8, 2752)]


def grad_inputs(shape, dtype, seed=0):
    gen = torch.Generator().manual_seed(sum(shape) + seed)
    rows = torch.exp(torch.randn(shape[0], 1, generator=gen))
    gate = (torch.randn(*shape, generator=gen) * 2 * rows).to(dtype)
    return (torch.randn(*shape, generator=gen) * 0.1).to(dtype), gate, (torch.randn(*shape, generator=gen) * rows).to(dtype)


def check_codes_near(got, scales, want, off, fmt):
    """Codes along the rows of `want`: scales and values within their rounding and `off`."""
    top = ref.blocks_amax(want, 1).t()
    top_off = ref.blocks_amax(off, 1).t()
    scales = scales.cpu().double()
    # the largest of values within `off` is within the largest `off`
    low = 2.0 ** -100 / ref.F8_MAX[fmt]
    within(scales, (top / ref.F8_MAX[fmt]).clamp_min(low), 1.001 * top_off / ref.F8_MAX[fmt] + 2 * U * scales)
    wide = ref.spread(scales, *want.shape)
    # half a step of a code: relative for a normal value, of the least step for a subnormal one
    half, least = (2.0 ** -4, 2.0 ** -10) if fmt == E4M3 else (2.0 ** -3, 2.0 ** -17)
    within(ref.values(down(got), scales), want, (half + 4 * U) * (want.abs() + off) + off + 1.001 * least * wide)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", GRAD_SHAPES)
def test_gated_grad(fp4q, shape, dtype, act):
    m, n = shape
    ins = grad_inputs(shape, dtype)
    for fmt in (E5M2, E4M3):
        got = fp4q.fp4q_gated8_backward(*(t.to(DEV) for t in ins), act, fmt, want_y=True)
        (dg, og), (du, ou), (y, oy) = gref.gated_grad(*ins, act)
        want, off = gref.join(dg, du), gref.join(og, ou)
        assert got.codes.dtype == got.codes_t.dtype == fmt and got.y_codes_t.dtype == E4M3
        assert got.codes.shape == want.shape and got.codes_t.shape == want.t().shape
        check_codes_near(got.codes, got.scales, want, off, fmt)
        check_codes_near(got.codes_t, got.scales_t, want.t(), off.t(), fmt)
        check_codes_near(got.y_codes_t, got.y_scales_t, y.t(), oy.t(), E4M3)
        pad = ref.groups(n) * 128
        assert bool((down(got.codes).float()[:, n:pad] == 0).all())
        assert bool((down(got.codes_t).float()[n:pad] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", GRAD_SHAPES)
def test_gated_grad_is_the_quantiser_of_the_joined_tensor(fp4q, shape, dtype):
    """With relu the gradients are products of the inputs: codes and scales exactly."""
    dy, gate, u = (t.float() for t in grad_inputs(shape, dtype, 1))
    got = fp4q.fp4q_gated8_backward(*(t.to(dtype).to(DEV) for t in (dy, gate, u)), "relu", want_y=True)
    whole = gref.join(torch.where(gate > 0, dy * u, 0.0), dy * gate.clamp_min(0.0))
    for c, s, want, fmt in ((got.codes, got.scales, whole, E5M2), (got.codes_t, got.scales_t, whole.t(), E5M2),
                            (got.y_codes_t, got.y_scales_t, (gate.clamp_min(0.0) * u).t(), E4M3)):
        values, scales = ref.quantize(want.contiguous(), fmt, False)
        assert same(s.cpu(), scales) and same(down(c).float(), values)


@pytest.mark.parametrize("ask", [(True, False, False), (False, True, False), (False, False, True), (True, False, True)])
def test_gated_grad_in_parts(fp4q, ask):
    ins = [t.to(DEV) for t in grad_inputs((200, 300), BF16)]
    whole = fp4q.fp4q_gated8_backward(*ins, "gelu", want_y=True)
    part = fp4q.fp4q_gated8_backward(*ins, "gelu", straight=ask[0], transposed=ask[1], want_y=ask[2])
    for i in range(3):
        if ask[i]:
            assert torch.equal(down(part[2 * i]).view(torch.uint8), down(whole[2 * i]).view(torch.uint8))
            assert torch.equal(part[2 * i + 1], whole[2 * i + 1])
        else:
            assert part[2 * i] is None and part[2 * i + 1] is None
    none = fp4q.fp4q_gated8_backward(*(torch.empty(0, 300, dtype=BF16, device=DEV) for _ in range(3)), want_y=True)
    assert none.codes.shape == (0, 684) and none.codes_t.shape == (684, 0) and none.y_scales_t.shape == (0, 300)


@pytest.mark.parametrize("act", ACTS)
def test_activations_at_their_ends(fp4q, act):
    """Gates from far below to far above, zeros of both signs, and what is not finite: every
    finite gate gives finite codes that are right, a NaN marks its own blocks."""
    g = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 3.0, -3.0, 8.0, -8.0, 15.9, 16.1, -15.9, -16.1, 79.0, -79.0, 81.0,
                      -81.0, 100.0, -100.0, 1e4, -1e4, 1e10, -1e10, 1e18, -1e18, 1e25, -1e25])
    gate = g.repeat(4, 5)[:, :130].contiguous()
    dy, u = torch.full_like(gate, 2.0 ** -40), torch.full_like(gate, 2.0 ** -30)
    got = fp4q.fp4q_gated8_backward(dy.to(DEV), gate.to(DEV), u.to(DEV), act, E4M3, want_y=True)
    (dg, og), (du, ou), (y, oy) = gref.gated_grad(dy, gate, u, act)
    want, off = gref.join(dg, du), gref.join(og, ou)
    check_codes_near(got.codes, got.scales, want, off, E4M3)
    check_codes_near(got.codes_t, got.scales_t, want.t(), off.t(), E4M3)
    check_codes_near(got.y_codes_t, got.y_scales_t, y.t(), oy.t(), E4M3)
    gate[1, 5] = float("nan")
    got = fp4q.fp4q_gated8_backward(dy.to(DEV), gate.to(DEV), u.to(DEV), act, E4M3, want_y=True)
    nan = torch.zeros(4, 386, dtype=torch.bool)
    nan[1, :128] = nan[1, 256:384] = True
    assert torch.equal(down(got.codes).float().isnan(), nan)
    nan = torch.zeros(386, 4, dtype=torch.bool)
    nan[5] = nan[261] = True
    assert torch.equal(down(got.codes_t).float().isnan(), nan)
    assert torch.equal(down(got.y_codes_t).float().isnan(), nan[256:])


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(fp4q, act):
    """Directional derivatives of sum(y dy) in 64 bits, central differences.  Columns of one row
    are blocks of one value, whose code is the largest one: the transposed codes hold dgate and
    dup to fp32."""
    gen = torch.Generator().manual_seed(11)
    n = 200
    dy, gate, u = (torch.randn(1, n, generator=gen) for _ in range(3))
    gate = torch.where(gate.abs() < 0.01, 0.5, gate)    # off relu's corner
    got = fp4q.fp4q_gated8_backward(dy.to(DEV), gate.to(DEV), u.to(DEV), act)
    both = ref.values(down(got.codes_t), got.scales_t.cpu()).t()
    dgate, dup = both[:, :n], both[:, -n:]

    def loss(g, u):
        return float((gref.activate(g, act)[0] * u * dy.double()).sum())

    step = 1e-4
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        vg, vu = torch.randn(1, n, generator=g).double(), torch.randn(1, n, generator=g).double()
        gd, ud = gate.double(), u.double()
        diff = (loss(gd + step * vg, ud + step * vu) - loss(gd - step * vg, ud - step * vu)) / (2 * step)
        size = float((dgate * vg).abs().sum() + (dup * vu).abs().sum())
        # the differences' own error is about step^2 = 1e-8 of the third derivatives
        assert abs(diff - float((dgate * vg).sum() + (dup * vu).sum())) <= (100 * U + 1e-6) * size


def test_gated_grad_past_32_bits(fp4q):
    rows, cols = 130048, 16512      # multiples of 128: 2.1e9 elements
    shape = (256, cols)
    part = [t.to(DEV) for t in grad_inputs(shape, BF16)]
    whole = []
    for t in part:
        w = torch.zeros(rows, cols, dtype=BF16, device=DEV)
        w[-256:] = t
        whole.append(w)
    want = fp4q.fp4q_gated8_backward(*part, "silu", want_y=True)
    got = fp4q.fp4q_gated8_backward(*whole, "silu", want_y=True)
    as_bytes = lambda t: t.view(torch.uint8)  # noqa: E731
    assert torch.equal(as_bytes(got.codes)[-256:], as_bytes(want.codes))
    assert torch.equal(got.scales[:, -256:], want.scales)
    assert torch.equal(as_bytes(got.codes_t)[:, -256:], as_bytes(want.codes_t))
    assert torch.equal(got.scales_t[-2:], want.scales_t)
    assert torch.equal(as_bytes(got.y_codes_t)[:, -256:], as_bytes(want.y_codes_t))
    assert torch.equal(got.y_scales_t[-2:], want.y_scales_t)


# -------------------------------------------------------------- 4-bit weights
GEMV_SHAPES = [(1, 1, 256), (1, 16, 512), (2, 17, 256), (1, 300, 4096), (3, 100, 1280), (5, 33, 11008), (6, 64, 4096),
               (8, 40, 2048), (16, 130, 4096), (17, 50, 768), (33, 20, 2560), (64, 48, 1024), (130, 70, 512), (1, 8, 16384),
               (4, 2752, 768)]


def weight(fp4q, n, k, flags, seed=0):
    gen = torch.Generator().manual_seed(n + k + seed)
    w = torch.randn(n, k, generator=gen) * torch.exp(torch.randn(n, 1, generator=gen)) * k ** -0.5
    return fp4q.fp4q_compress(w.to(BF16).to(DEV), flags=flags)


def rows(m, k, dtype, seed=0):
    gen = torch.Generator().manual_seed(m + k + seed)
    x = torch.randn(m, k, generator=gen) * torch.exp(torch.randn(m, 1, generator=gen))
    x[:, ::97] *= 30
    return x.to(dtype)


def parts_of(dtype, out_dtype, plain):
    """One part where transformed bf16 x has bf16 out; two (of which the second may be zeros) else."""
    return 1 if not plain and dtype == out_dtype == BF16 else 2


@pytest.mark.parametrize("shape", GEMV_SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("plain", [True, False])
def test_gemv4(fp4q, shape, dtype, plain):
    print(shape, dtype, plain, flush=True)
    m, n, k = shape
    flags = fp4q.FP4Q_FLAG_NO_FWHT if plain else 0
    w, x = weight(fp4q, n, k, flags), rows(m, k, dtype)
    for out_dtype in (F32, BF16):
        want, off = gref.gemv4(x, w, not plain, parts_of(dtype, out_dtype, plain))
        got = fp4q.fp4q_gemv4(x.to(DEV), w, flags, out_dtype=out_dtype)
        assert got.dtype == out_dtype and got.shape == (m, n)
        within(got.cpu(), want, off + (HALF_STEP[BF16] * (want.abs() + off) if out_dtype == BF16 else 0))
    assert fp4q.fp4q_gemv4(x.to(DEV), w, flags).dtype == dtype
    out = torch.full((m, n), float("nan"), dtype=out_dtype, device=DEV)
    assert fp4q.fp4q_gemv4(x.to(DEV), w, flags, out=out) is out and torch.equal(out, got)


@pytest.mark.parametrize("shape", GEMV_SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("plain", [True, False])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gated4(fp4q, shape, dtype, plain, act):
    print(shape, dtype, plain, act, flush=True)
    m, n, k = shape
    flags = fp4q.FP4Q_FLAG_NO_FWHT if plain else 0
    gate, u, x = weight(fp4q, n, k, flags), weight(fp4q, n, k, flags, 1), rows(m, k, dtype)
    for out_dtype in (F32, BF16):
        (g, off_g), (v, off_v) = (gref.gemv4(x, w, not plain, parts_of(dtype, out_dtype, plain)) for w in (gate, u))
        value, slope, off, _ = gref.activate(g, act)
        off = off + off_g * (1.2 + off_g)
        want, off = value * v, off * (v.abs() + off_v) + value.abs() * off_v
        got = fp4q.fp4q_gated4(x.to(DEV), gate, u, act, flags, out_dtype=out_dtype)
        assert got.dtype == out_dtype and got.shape == (m, n)
        within(got.cpu(), want, off + 2 * U * want.abs() + (HALF_STEP[BF16] * (want.abs() + off) if out_dtype == BF16 else 0))
    assert fp4q.fp4q_gated4(x.to(DEV), gate, u, act, flags).dtype == dtype


def test_payload_values_are_the_receivers(fp4q):
    """The references' weight is what the receiver makes of the payload."""
    for flags in (0, fp4q.FP4Q_FLAG_NO_FWHT):
        w = weight(fp4q, 20, 1024, flags)
        v = gref.payload_values(w)
        if not flags:
            v = (v.view(20, -1, 256) @ gref.hadamard()).view(20, -1) / 16
        got = fp4q.fp4q_decompress(*w, flags=flags).cpu()
        within(got, v, 12 * U * v.abs().view(20, -1, 256).amax(dim=2).repeat_interleave(256, 1) * 16)


@pytest.mark.parametrize("m", [1, 5, 20])
@pytest.mark.parametrize("plain", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_few_rows_carry_what_is_not_finite(fp4q, m, plain, dtype):
    """A NaN or an infinity in x reaches its own row, and no other."""
    flags = fp4q.FP4Q_FLAG_NO_FWHT if plain else 0
    w, x = weight(fp4q, 40, 1024, flags), rows(m, 1024, dtype)
    for bad in (float("nan"), float("inf")):
        x[m - 1, 300] = bad
        for got in (fp4q.fp4q_gemv4(x.to(DEV), w, flags), fp4q.fp4q_gated4(x.to(DEV), w, w, flags=flags)):
            assert not bool(got[m - 1].isfinite().any()) if bad != bad else not bool(got[m - 1].isfinite().all())
            assert bool(got[:m - 1].isfinite().all())


@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** -90])
@pytest.mark.parametrize("plain", [True, False])
def test_few_rows_far_from_one(fp4q, scale, plain):
    """Values of x near the ends of what may be given: the parts and the blocks' sums keep
    their range."""
    flags = fp4q.FP4Q_FLAG_NO_FWHT if plain else 0
    w, x = weight(fp4q, 40, 512, flags), rows(3, 512, F32) * scale
    # parts of x below 2^-112 may be dropped (its power of two is at most 2^98), and of a
    # block's sum what lies below 2^-126 before its scale times 2^17
    low = 512 * 2.0 ** -112 * float(gref.payload_values(w).abs().max()) + 2 * 2.0 ** -109 * float(w[2].max())
    want, off = gref.gemv4(x, w, not plain)
    within(fp4q.fp4q_gemv4(x.to(DEV), w, flags).cpu(), want, off + low)
    if scale > 1:
        x = torch.where(x > 0, 1.0, -1.0) * 2.0 ** 118 * (1 - 2.0 ** -24)
        want, off = gref.gemv4(x, w, not plain)
        within(fp4q.fp4q_gemv4(x.to(DEV), w, flags).cpu(), want, off + low)


def test_few_rows_of_nothing(fp4q):
    w = weight(fp4q, 40, 512, 0)
    assert fp4q.fp4q_gemv4(torch.empty(0, 512, device=DEV), w).shape == (0, 40)
    assert fp4q.fp4q_gated4(torch.empty(0, 512, device=DEV), w, w).shape == (0, 40)
    none = tuple(t[:0] for t in w)
    assert fp4q.fp4q_gemv4(torch.ones(3, 512, device=DEV), none).shape == (3, 0)
    zero = tuple(torch.zeros_like(t) for t in w)
    assert bool((fp4q.fp4q_gemv4(torch.ones(3, 512, device=DEV), zero) == 0).all())


def test_gemv4_past_32_bits(fp4q):
    """A payload whose codes take more than 4 GiB: its last rows against those alone."""
    n, k = 800000, 11008
    flags = fp4q.FP4Q_FLAG_NO_FWHT
    part, x = weight(fp4q, 50, k, flags), rows(2, k, BF16).to(DEV)
    whole = []
    for t in part:
        w = torch.zeros(n, t.shape[1], dtype=t.dtype, device=DEV)
        w[-50:] = t
        whole.append(w)
    want = fp4q.fp4q_gemv4(x, part, flags)
    got = fp4q.fp4q_gemv4(x, tuple(whole), flags)
    assert torch.equal(got[:, -50:], want) and bool((got[:, :-50] == 0).all())
    got = fp4q.fp4q_gated4(x, tuple(whole), tuple(whole), flags=flags)
    assert torch.equal(got[:, -50:], fp4q.fp4q_gated4(x, part, part, flags=flags)) and bool((got[:, :-50] == 0).all())


# ------------------------------------------ together, on streams and in graphs
def training(fp4q, x, weight_norm, gate_up, down_w, d, act, stream=None):
    """A gated layer behind a norm, forward and backward, with the 8-bit linear-layer operators."""
    norm = fp4q.fp4q_rmsnorm(x, weight_norm, 1e-6, want_codes=True, want_rstd=True, stream=stream)
    h = fp4q.fp4q_gated8(norm.codes, norm.scales, gate_up.codes, gate_up.scales, act, want_pre=True, stream=stream)
    q = fp4q.fp4q_quantize8(h.y, stream=stream)
    out = fp4q.fp4q_gemm8(q.codes, q.scales, down_w.codes, down_w.scales, stream=stream)
    qd = fp4q.fp4q_quantize8(d, E5M2, transposed=True, stream=stream)
    dy = fp4q.fp4q_gemm8(qd.codes, qd.scales, down_w.codes_t, down_w.scales_t, stream=stream)
    g = fp4q.fp4q_gated8_backward(dy, h.gate, h.up, act, want_y=True, stream=stream)
    x_t = fp4q.fp4q_quantize8(norm.y, straight=False, transposed=True, stream=stream)
    dn = fp4q.fp4q_gemm8(g.codes, g.scales, gate_up.codes_t, gate_up.scales_t, stream=stream)
    dgu = fp4q.fp4q_gemm8(g.codes_t, g.scales_t, x_t.codes_t, x_t.scales_t, out_dtype=F32, stream=stream)
    ddown = fp4q.fp4q_gemm8(qd.codes_t, qd.scales_t, g.y_codes_t, g.y_scales_t, out_dtype=F32, stream=stream)
    dx, dw = fp4q.fp4q_rmsnorm_backward(dn, norm.h, weight_norm, norm.rstd, stream=stream)
    return [out, dx, dw, dgu, ddown]


def layer_inputs(fp4q, tokens, hidden, inner, seed=0):
    gen = torch.Generator().manual_seed(tokens + seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    gate, u = rand(inner, hidden) * hidden ** -0.5, rand(inner, hidden) * hidden ** -0.5
    down_w = (rand(hidden, inner) * inner ** -0.5).to(BF16)
    joined_w = gref.join(gate.t(), u.t()).t().contiguous().to(BF16)
    x, d, w = rand(tokens, hidden).to(BF16), (0.1 * rand(tokens, hidden)).to(BF16), (1 + 0.1 * rand(hidden)).to(BF16)
    return x, w, joined_w, down_w, d


@pytest.mark.parametrize("tokens,hidden,inner", [(7, 256, 200), (96, 512, 1024), (300, 520, 333)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_a_gated_layer_together(fp4q, tokens, hidden, inner, act):
    """Forward and backward against fp32 autograd on the CPU.  An 8-bit operand is off by at
    most 2^-4 (E4M3) or 2^-3 (E5M2) of a value, which random values average to at most 0.04 and
    0.08 of a product's norm; the layer chains two products with a product of two between (both
    off: twice the first one's error) and as many back."""
    x, w, joined_w, down_w, d = layer_inputs(fp4q, tokens, hidden, inner)
    q = [fp4q.fp4q_quantize8(t.to(DEV), tiles=True, transposed=True) for t in (joined_w, down_w)]
    got = training(fp4q, x.to(DEV), w.to(DEV), q[0], q[1], d.to(DEV), act)
    xs, ws, js, ds = (t.float().requires_grad_() for t in (x, w, joined_w, down_w))
    h = xs * torch.rsqrt(xs.square().mean(dim=1, keepdim=True) + 1e-6) * ws
    p = ref.groups(inner) * 128
    gate, u = h @ js[:inner].t(), h @ js[p:].t()
    value = torch.nn.functional.silu(gate) if act == "silu" else torch.nn.functional.gelu(gate, approximate="tanh")
    out = (value * u) @ ds.t()
    (out * d.float()).sum().backward()
    for name, a, b in zip(("out", "dx", "dw", "djoined", "ddown"), got, (out.detach(), xs.grad, ws.grad, js.grad, ds.grad)):
        off = float((a.cpu().float() - b).norm() / b.norm())
        print(name, off, flush=True)
        assert off < 0.2, name
    assert bool((got[3][inner:p] == 0).all())    # the joined weight's padding rows get no gradient


@pytest.mark.parametrize("tokens", [3, 200])
def test_training_on_streams_and_in_graphs(fp4q, tokens):
    """The same values on another stream and from a graph, replayed among eager work."""
    x, w, joined_w, down_w, d = (t.to(DEV) for t in layer_inputs(fp4q, tokens, 520, 300))
    q = [fp4q.fp4q_quantize8(t, tiles=True, transposed=True) for t in (joined_w, down_w)]
    run = lambda stream=None: training(fp4q, x, w, q[0], q[1], d, "silu", stream)  # noqa: E731
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = run()
    for turn in range(4):
        x.copy_(layer_inputs(fp4q, tokens, 520, 300, turn + 1)[0].to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(run(), held)), turn


@pytest.mark.parametrize("ranks,tokens,hidden,inner", [(2, 96, 512, 1024), (4, 7, 256, 528), (1, 200, 512, 300)])
def test_example_layer_gated(fp4q, ranks, tokens, hidden, inner):
    """The gated layer of examples/tp_layer.py against fp32: the bounds of the two products above,
    and FP4's 0.15 in the norm at each of two exchanges."""
    from examples import tp_layer
    plain = tp_layer.errors(ranks, tokens, hidden, inner, compress=False, gated=True)
    fp4 = tp_layer.errors(ranks, tokens, hidden, inner, compress=True, gated=True)
    print(plain, fp4, flush=True)
    assert max(plain.values()) < 0.2
    assert max(fp4.values()) < 0.5


def test_example_token(fp4q):
    """A 4-bit weight is off by at most 0.25 of a value, 0.15 in the norm, of a product as much;
    the activation's product doubles it and the second projection adds its own."""
    from examples import tp_layer
    assert tp_layer.token_error(2, 3, 512, 1024) < 0.5
    assert tp_layer.token_error(2, 1, 512, 600) < 0.5    # a shard of 300: padded


def serving(fp4q, x, w, gate, u, down_w, flags, stream=None):
    """One step of single tokens through the same layer with 4-bit weights."""
    n = fp4q.fp4q_rmsnorm(x, w, 1e-6, stream=stream).y
    h = fp4q.fp4q_gated4(n, gate, u, flags=flags, stream=stream)
    return [fp4q.fp4q_gemv4(h, down_w, flags=flags, stream=stream)]


@pytest.mark.parametrize("tokens", [1, 9])
@pytest.mark.parametrize("plain", [True, False])
def test_serving_with_4_bit_weights(fp4q, tokens, plain):
    """Against the same layer in 64 bits on the payloads' values, on a stream, and in a graph
    that is replayed among eager work."""
    flags, hidden, inner = (fp4q.FP4Q_FLAG_NO_FWHT if plain else 0), 1024, 768
    ws = [weight(fp4q, *s, flags, i) for i, s in enumerate([(inner, hidden), (inner, hidden), (hidden, inner)])]
    x, w = rows(tokens, hidden, BF16).to(DEV), torch.ones(hidden, dtype=BF16, device=DEV)
    got = serving(fp4q, x, w, *ws, flags)[0]
    y = ref.norm(x.cpu(), w.cpu(), 1e-6)[1]
    g, u = (gref.gemv4(y, p, not plain)[0] for p in ws[:2])
    want = gref.gemv4(gref.activate(g, "silu")[0] * u, ws[2], not plain)[0]
    # three roundings to bf16 (2^-8 each at most, the gated product's input counted in both
    # factors) that random values average: 0.01 of the norm and more would be another error
    assert float((got.cpu().double() - want).norm()) <= 0.01 * float(want.norm())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = serving(fp4q, x, w, *ws, flags, side)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, on_side)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = serving(fp4q, x, w, *ws, flags)[0]
    for turn in range(4):
        x.copy_(rows(tokens, hidden, BF16, turn + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(serving(fp4q, x, w, *ws, flags)[0], held), turn
