"""Plain references of the 8-bit linear-layer operators for the tests, in 64 bits,
and the bounds of what fp32 kernels may be off by (u = 2^-24, half a step of fp32)."""
import torch

U = 2.0 ** -24
GROUP = 128
F8_MAX = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
HALF_STEP = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
# Longest chain of additions behind one sum over a row: 64 values a lane, then 6 steps
# over the lanes and at most 16 over the wavefronts.
ROW_CHAIN = 64 + 6 + 16


def groups(n):
    return (n + GROUP - 1) // GROUP


def blocks_amax(v, rows_per_block):
    """Largest magnitude of each block of rows_per_block x 128 -> [row blocks, groups]."""
    r, c = v.shape
    gr, gc = -(-r // rows_per_block), groups(c)
    pad = torch.zeros(gr * rows_per_block, gc * GROUP, dtype=v.dtype)
    pad[:r, :c] = v.abs()
    return pad.view(gr, rows_per_block, gc, GROUP).amax(dim=(1, 3))


def quantize(v, fmt, tiles):
    """Codes (as fp32 values) and scales by the definition, on fp32 values: exact."""
    per = GROUP if tiles else 1
    top = blocks_amax(v, per)
    scale = top.clamp_min(2.0 ** -100) / F8_MAX[fmt]
    scale = torch.where(torch.isfinite(top), scale, torch.full_like(scale, float("nan")))
    wide = scale.repeat_interleave(per, 0)[:v.shape[0]].repeat_interleave(GROUP, 1)[:, :v.shape[1]]
    return (v / wide).to(fmt).float(), scale.t().contiguous()


def spread(scales, rows, k):
    """Scales [groups, rows or row tiles] as fp64 [rows, k]."""
    s = scales.double().t()
    if s.shape[0] != rows:
        s = s.repeat_interleave(GROUP, 0)[:rows]
    return s.repeat_interleave(GROUP, 1)[:, :k]


def values(codes, scales):
    return codes.float().double() * spread(scales, codes.shape[0], codes.shape[1])


def norm(h, w, eps):
    """rstd and y in 64 bits of the stored h."""
    h, w = h.double(), w.double()
    r = 1.0 / torch.sqrt((h * h).mean(dim=1) + eps)
    return r, h * r[:, None] * w


def norm_grad(dy, h, w, r, dh):
    """dx, dw in 64 bits and bounds of their fp32 evaluation."""
    dy, h, w, r = dy.double(), h.double(), w.double(), r.double()
    g, xhat = dy * w, h * r[:, None]
    m = (g * xhat).mean(dim=1, keepdim=True)
    dx = r[:, None] * (g - xhat * m)
    # g, xhat one rounding each; the mean's chain, its products and its division; the
    # outer product, difference and scaling
    spread_m = (g * xhat).abs().mean(dim=1, keepdim=True)
    off = r[:, None] * U * (4 * g.abs() + xhat.abs() * ((ROW_CHAIN + 6) * spread_m + 4 * m.abs()))
    if dh is not None:
        dx = dx + dh.double()
    dw = (dy * xhat).sum(dim=0)
    dw_off = (dy * xhat).abs().sum(dim=0) * U * (h.shape[0] + 3)
    return dx, off + U * dx.abs(), dw, dw_off


def gemm(a, sa, b, sb):
    """The product in 64 bits and the bound of its fp32 evaluation (fp32 output): 128
    additions of a block (a whole step each, whatever way the matrix core rounds), two
    for its scale, one for each block and a split's join."""
    va, vb = values(a, sa), values(b, sb)
    n = sa.shape[0]
    return va @ vb.t(), (va.abs() @ vb.abs().t()) * U * (2 * GROUP + n + 8)


def gemm_bf16_off(a, sa, b, sb, want):
    """The bound of the product with bf16 output: of 8 neighbouring products the matrix
    core drops what lies below 2^-13 of the largest, from at most 7 of them; then half a
    step of bf16."""
    sums = values(a, sa).abs() @ values(b, sb).abs().t()
    off = sums * (7 * 2.0 ** -13 + U * (2 * GROUP + sa.shape[0] + 8))
    return off + HALF_STEP[torch.bfloat16] * (want.abs() + off)


def fake_codes(gen, rows, cols, fmt, pad=0x7F):
    """Random codes whose rows are padded to 16 bytes with NaN codes."""
    pitch = (cols + 15) // 16 * 16
    room = torch.full((rows, pitch), pad, dtype=torch.uint8)
    room[:, :cols] = torch.randn(rows, cols, generator=gen).mul(8).to(fmt).view(torch.uint8)
    return room.view(fmt)[:, :cols]
