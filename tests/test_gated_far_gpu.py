"""The gated operators where the gate is far from zero: the activations take their limits, whatever
fp32 number or infinity the gate is, in the gradients and in the products."""
import pytest

torch = pytest.importorskip("torch")

from tests import gated_ref as gref
from tests import linear_ref as ref
from tests.linear_ref import HALF_STEP, U
from tests.test_gated_gpu import ACTS, BF16, DEV, E4M3, F32
from tests.test_linear_gpu import down, fp4q, within  # noqa: F401 (fp4q is the fixture)

pytestmark = pytest.mark.gpu
INF = float("inf")
# a bf16 is among the fp32 numbers: both types hold each of these exactly
FAR = [float(torch.tensor(v).to(BF16)) for v in (88.0, 96.0, 130.0, 1e5, 1e19, 1e28, 1e30, 1e33, 1e36, 3.38e38)]


def one_row(got, n):
    """dgate, dup and y of one row from the transposed codes, whose blocks are single values: the
    largest code times the scale holds each to fp32."""
    both = ref.values(down(got.codes_t), got.scales_t.cpu()).t()
    return both[:, :n], both[:, -n:], ref.values(down(got.y_codes_t), got.y_scales_t.cpu()).t()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("up", [1.0, -2.0 ** -20])
def test_gradients_of_far_gates(fp4q, act, dtype, up):
    """Beyond 88 the logistic and the normal distribution are 0 or 1 to 2^-126: the activation is g
    or 0 and its derivative 1 or 0.  Of the result g times 2^-126 may remain, not more; a value
    below 2^-100 counts as that for its scale, and its code is off by half the least step of it."""
    gate = torch.tensor([FAR + [-v for v in FAR]], dtype=dtype)
    assert torch.equal(gate.float(), torch.tensor([FAR + [-v for v in FAR]]))
    dy, u = torch.full_like(gate, 0.5), torch.full_like(gate, up)
    got = fp4q.fp4q_gated8_backward(*(t.to(DEV) for t in (dy, gate, u)), act, E4M3, want_y=True)
    g = gate.double()
    on = (g > 0).double()
    left = g.abs() * 2.0 ** -126
    for value, want, factor in zip(one_row(got, gate.shape[1]), (0.5 * up * on, 0.5 * on * g, up * on * g),
                                   (abs(0.5 * up), 0.5, abs(up))):
        # three products, the scale's quotient and the codes' product with it: a rounding each
        within(value, want, 8 * U * want.abs() + factor * left + 2.0 ** -100 / 448 * 2.0 ** -10)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_of_an_infinite_gate(fp4q, act, dtype):
    """Far below, everything is 0; far above the derivative is 1, and what the activation itself
    is a factor of is infinite: no scale holds it."""
    gate = torch.tensor([[INF, -INF, 1.0]], dtype=dtype)
    dy, u = torch.full_like(gate, 0.5), torch.full_like(gate, 3.0)
    got = fp4q.fp4q_gated8_backward(*(t.to(DEV) for t in (dy, gate, u)), act, E4M3, want_y=True)
    dgate, dup, y = one_row(got, 3)
    assert abs(float(dgate[0, 0]) - 1.5) <= 8 * U * 1.5 and float(dgate[0, 1]) == 0
    assert bool(dup[0, 0].isnan()) and float(dup[0, 1]) == 0
    assert bool(y[0, 0].isnan()) and float(y[0, 1]) == 0
    assert bool(torch.stack([dgate[0, 2], dup[0, 2], y[0, 2]]).isfinite().all())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [1, 16, 40, 300, 2100])
@pytest.mark.parametrize("power", [45, 55, 63, 75])
def test_products_of_far_gates(fp4q, act, m, power):
    """Gates of 2^(2 power) and of minus that, from scales of 2^power on both sides of the first
    block (2^150 is an infinity), and ups from the second: y is the gate times the up, or 0."""
    n, k = 200, 256
    a = torch.zeros(m, k)
    a[:, 0] = torch.where(torch.arange(m) % 2 == 0, 1.0, -1.0)
    a[:, 128] = 1.0
    p = ref.groups(n) * 128
    w = torch.zeros(p + n, k)
    w[:n, 0] = torch.where(torch.arange(n) % 3 == 0, -1.0, 1.0)
    w[p:, 128] = torch.where(torch.arange(n) % 5 == 0, -0.5, 1.5)
    sa, sw = torch.ones(2, m), torch.ones(2, 2 * ref.groups(n))
    sa[0], sw[0] = 2.0 ** power, 2.0 ** power
    got = fp4q.fp4q_gated8(a.to(E4M3).to(DEV), sa.to(DEV), w.to(E4M3).to(DEV), sw.to(DEV), act, want_pre=True)
    sign = a[:, :1].double() * w[:n, 0].double()
    gate = sign * (2.0 ** (2 * power) if 2 * power < 128 else INF)
    up = w[p:, 128].double().expand(m, n)
    assert torch.equal(got.gate.cpu().double(), gate) and torch.equal(got.up.cpu().double(), up)
    y = got.y.cpu().double()
    want = torch.where(sign > 0, gate * up, 0.0)
    assert bool((y[sign < 0].abs() <= 2.0 ** (2 * power - 126) if 2 * power < 128 else y[sign < 0] == 0).all())
    assert torch.equal(y[sign > 0], want[sign > 0])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [1, 5, 20])
@pytest.mark.parametrize("power", [40, 65])
def test_few_rows_of_far_gates(fp4q, act, m, power):
    """The 4-bit form: gates of about 2^(2 power) with both signs (2^130 is an infinity)."""
    n, k, flags = 48, 512, fp4q.FP4Q_FLAG_NO_FWHT
    w, v = torch.zeros(n, k), torch.zeros(n, k)
    w[:, 3] = torch.where(torch.arange(n) % 3 == 0, -1.0, 1.0) * 2.0 ** power
    v[:, 300] = 1.5
    x = torch.zeros(m, k)
    x[:, 3], x[:, 300] = 2.0 ** power, 0.5
    gate, up = (fp4q.fp4q_compress(t.to(BF16).to(DEV), flags=flags) for t in (w, v))
    got = fp4q.fp4q_gated4(x.to(DEV), gate, up, act, flags).cpu().double()
    sign = w[:, 3].sign().double().expand(m, n)
    big = x[:, 3:4].double() @ gref.payload_values(gate)[:, 3:4].t()
    u = (x.double() @ gref.payload_values(up).t())
    assert bool((got[sign < 0].abs() <= 2.0 ** (2 * power - 126) if 2 * power < 128 else got[sign < 0] == 0).all())
    if 2 * power < 128:
        within(got[sign > 0], (big * u)[sign > 0], 16 * U * (big * u).abs()[sign > 0])
    else:
        assert bool((got[sign > 0] == INF).all())


@pytest.mark.parametrize("act", ACTS)
def test_products_near_the_end_of_the_exponential(fp4q, act):
    """Gates from -72 to -112, where exp(-g) leaves fp32's range, against 64 bits: what lies below
    2^-126 of the gate may count as 0."""
    n, k = 41, 256
    a = torch.zeros(1, k)
    a[0, 0] = a[0, 128] = 1.0
    p = ref.groups(n) * 128
    w = torch.zeros(p + n, k)
    # eight times 9 to 14, which codes hold
    g = torch.tensor([-float(c) for c in (72, 80, 88, 96, 104, 112)])
    w[:6, 0], w[p:p + 6, 128] = g / 8, 1.0
    sa, sw = torch.ones(2, 1), torch.ones(2, 2)
    sa[0] = 8.0
    got = fp4q.fp4q_gated8(a.to(E4M3).to(DEV), sa.to(DEV), w.to(E4M3).to(DEV), sw.to(DEV), act, want_pre=True)
    assert torch.equal(got.gate.cpu()[0, :6].float(), g)
    value = gref.activate(g.double(), act)[0]
    steps = 24 + 6 * 2 * g.double() ** 2        # as in the reference: of e^z its argument's rounding, z^2 at most
    within(got.y.cpu()[0, :6], value, (HALF_STEP[BF16] + U * steps) * value.abs() + g.double().abs() * 2.0 ** -126)
