"""Plain references of the gated operators for the tests, in 64 bits, and the bounds of what
fp32 kernels may be off by (U = 2^-24, half a step of fp32)."""
import torch

from tests import linear_ref as ref
from tests.linear_ref import U

ACTS = ("silu", "gelu", "gelu_tanh", "relu")
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
C, D = (2 / torch.pi) ** 0.5, 0.044715


def activate(g, kind):
    """The activation and its derivative at 64-bit values, and bounds of their fp32 evaluation.

    Of e^z an error of z (a few roundings of its own) becomes |z| times as many; the rest is a
    handful of roundings and the hardware's 2^x, 1/x (1 unit each) and, for gelu, a fitted
    polynomial of degree 9 (16 units allowed for it and its argument).
    Where z is held at 80 a value differs by at most e^-80 (2^-115) of g."""
    far = g.abs() * 2.0 ** -115
    if kind == "relu":
        on = (g > 0).double()
        return g.clamp_min(0.0), on, torch.zeros_like(g), torch.zeros_like(g)
    if kind == "gelu":
        cdf = 0.5 * torch.erfc(-g * 0.5 ** 0.5)
        dens = torch.exp(-0.5 * g * g) * (0.5 / torch.pi) ** 0.5
        steps = 24 + 2 * g * g
        return (g * cdf, cdf + g * dens, U * steps * (g * cdf).abs() + far,
                U * steps * (cdf + (g * dens).abs()) + far)
    z, dz, err = g, torch.ones_like(g), 2.0
    if kind == "gelu_tanh":
        z, dz, err = 2 * C * (g + D * g ** 3), 2 * C * (1 + 3 * D * g * g), 6.0
    p, q = torch.special.expit(z), torch.special.expit(-z)
    steps = 24 + err * z.abs()
    return (g * p, p + g * dz * p * q, U * steps * (g * p).abs() + far,
            U * steps * (p + (g * dz * p * q).abs()) + far)


def gated_grad(dy, gate, up, kind):
    """dgate, dup and y in 64 bits of the given tensors, each with its bound."""
    dy, gate, up = dy.double(), gate.double(), up.double()
    act, slope, act_off, slope_off = activate(gate, kind)
    out = []
    for value, off in ((dy * up * slope, (dy * up).abs() * slope_off), (dy * act, dy.abs() * act_off),
                       (act * up, up.abs() * act_off)):
        out.append((value, off + 2 * U * value.abs() + 2.0 ** -140))
    return out


def join(gate, up):
    """[gate | 0 | up], the second half from a multiple of 128 on."""
    rows, n = gate.shape
    return torch.cat([gate, gate.new_zeros(rows, -n % ref.GROUP), up], dim=1)


def hadamard():
    h = torch.ones(1, 1, dtype=torch.float64)
    while h.shape[0] < 256:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def payload_values(payload):
    """The values of a payload's codes with both scales, without the transform, in 64 bits (exact)."""
    codes, micro, block = (t.cpu() for t in payload)
    n, half = codes.shape
    c = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(n, 2 * half).long()
    v = E2M1[c & 7] * (1 - 2 * (c >> 3)).double()
    v = v * micro.contiguous().view(torch.float8_e4m3fn).float().double().repeat_interleave(16, 1)
    return v * block.double().repeat_interleave(256, 1)


def gemv4(x, payload, transformed, parts=2):
    """x times the payload's weight, transposed, in 64 bits, and the bound of the kernel's fp32
    sum: 256 additions of a block and three parts (a whole step each, whatever way the matrix
    core rounds), the block's scale, an addition a block and the join of 16 wavefronts.  A
    transformed weight is H Q / 16: x is transformed in fp32 instead, eight stages of one
    rounding each on sums of at most the block's |x|, and a multiplication by 1/16 (exact).
    As fp16 under its block's power of two, the largest at 2^14 or more: a part that is a
    normal number is within 2^-11 of its value, two parts within 2^-22 (one part only where
    transformed bf16 x has bf16 out); a part below 2^-14 may count as zero, 2^-28 of the largest."""
    q, x = payload_values(payload), x.double().cpu()
    m, k = x.shape
    off_x = torch.zeros_like(x)
    if transformed:
        spread = x.abs().view(m, -1, 256).sum(dim=2).repeat_interleave(256, 1) / 16
        off_x = 8 * U * spread
        x = (x.view(m, -1, 256) @ hadamard()).reshape(m, k) / 16
    top = x.abs().view(m, -1, 256).amax(dim=2).repeat_interleave(256, 1)
    off_x = off_x + (4 * U if parts == 2 else 2.0 ** -11) * x.abs() + 2.0 ** -28 * top
    want = x @ q.t()
    return want, (x.abs() @ q.abs().t()) * U * (2 * 256 + k // 256 + 16 + 8) + off_x @ q.abs().t()
