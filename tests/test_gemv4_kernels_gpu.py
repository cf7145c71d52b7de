"""Every kernel of the 4-bit products, with one unit of outputs a workgroup and with several, against
64 bits."""
import pytest

torch = pytest.importorskip("torch")

from tests import gated_ref as gref
from tests import gemv4_shapes
from tests.linear_ref import HALF_STEP, U
from tests.test_gated_gpu import BF16, DEV, F32, parts_of
from tests.test_linear_gpu import fp4q, within  # noqa: F401 (fp4q is the fixture)

pytestmark = pytest.mark.gpu
TYPE = {gemv4_shapes.BF16: BF16, gemv4_shapes.F32: F32}


def weight(fp4q, gen, n, k, flags):
    w = torch.randn(n, k, generator=gen, device=DEV) * torch.exp(torch.randn(n, 1, generator=gen, device=DEV)) * k ** -0.5
    return fp4q.fp4q_compress(w.to(BF16), flags=flags)


def exact(x, payload, transformed, parts):
    """gated_ref.gemv4, value and bound, computed on the GPU."""
    codes, micro, block = payload
    n, k = codes.shape[0], 2 * codes.shape[1]
    c = torch.stack([codes & 15, codes >> 4], dim=-1).view(n, k).long()
    q = gref.E2M1.to(DEV)[c & 7] * (1 - 2 * (c >> 3)).double()
    q *= micro.view(torch.float8_e4m3fn).float().double().repeat_interleave(16, 1) * block.double().repeat_interleave(256, 1)
    x = x.double()
    off_x = torch.zeros_like(x)
    if transformed:
        off_x = 8 * U * x.abs().view(x.shape[0], -1, 256).sum(dim=2).repeat_interleave(256, 1) / 16
        x = torch.matmul(x.view(-1, 256), gref.hadamard().to(DEV)).view(x.shape) / 16
    top = x.abs().view(x.shape[0], -1, 256).amax(dim=2).repeat_interleave(256, 1)
    off_x = off_x + (4 * U if parts == 2 else 2.0 ** -11) * x.abs() + 2.0 ** -28 * top
    size = q.abs()
    return torch.matmul(x, q.t()), torch.matmul(x.abs(), size.t()) * U * (2 * 256 + k // 256 + 16 + 8) + torch.matmul(off_x, size.t())


@pytest.mark.parametrize("shape", gemv4_shapes.SHAPES)
def test_every_kernel(fp4q, shape):
    print(shape, flush=True)
    m, n, k, bits, transformed, gated, *want_plan = shape
    assert [gemv4_shapes.plan(m, n, k, bits, bits, transformed, gated)[i] for i in (0, 1, 4)] == want_plan
    dtype, flags = TYPE[bits], 0 if transformed else fp4q.FP4Q_FLAG_NO_FWHT
    gen = torch.Generator(device=DEV).manual_seed(m + n + k)
    x = torch.randn(m, k, generator=gen, device=DEV) * torch.exp(torch.randn(m, 1, generator=gen, device=DEV))
    x[:, ::97] *= 30
    x = x.to(dtype)
    weights = [weight(fp4q, gen, n, k, flags) for _ in range(1 + gated)]
    for out_dtype in (dtype, F32 if dtype == BF16 else BF16):
        want, off = exact(x, weights[0], transformed, parts_of(dtype, out_dtype, not transformed))
        if gated:
            u, off_u = exact(x, weights[1], transformed, parts_of(dtype, out_dtype, not transformed))
            value, _, act_off, _ = gref.activate(want, "silu")
            # the derivative is at most 1.2, its change at most 1 for a change of 1 in the gate
            off = act_off + off * (1.2 + off)
            want, off = value * u, off * (u.abs() + off_u) + value.abs() * off_u + 2 * U * (value * u).abs()
            call = lambda: fp4q.fp4q_gated4(x, *weights, "silu", flags, out_dtype=out_dtype)  # noqa: E731
        else:
            call = lambda: fp4q.fp4q_gemv4(x, weights[0], flags, out_dtype=out_dtype)  # noqa: E731
        got = call()
        assert got.dtype == out_dtype and got.shape == (m, n)
        within(got, want, off + (HALF_STEP[BF16] * (want.abs() + off) if out_dtype == BF16 else 0))
        assert torch.equal(got, call())
