"""One tensor-parallel MLP layer, forward and backward, with the ranks of one group emulated
in turn on one GPU: what leaves a rank is FP4-compressed, what a rank computes runs on 8-bit
operands with a scale per 128.

    python examples/tp_layer.py [--ranks 4] [--tokens 2048] [--hidden 4096] [--inner 11008] [--gated]

Forward, on every rank (its weight shards: up [inner / ranks, hidden], down
[hidden, inner / ranks]):
    payloads of the layer before --fp4q_decompress_accumulate--> x
    x + residual --fp4q_rmsnorm--> h, y, 8-bit codes of y
    codes, up    --fp4q_gemm8--> u,   a = max(u, 0)^2 --fp4q_quantize8--> 8-bit a
    a, down      --fp4q_gemm8--> this rank's part --fp4q_compress--> payload
Backward, from the gradient of the layer's output (the same on every rank):
    d, down^T --fp4q_gemm8--> da -> du;   du, up^T --fp4q_gemm8--> part of dy --> payload
    payloads --> dy --fp4q_rmsnorm_backward--> dx, dweight
    d^T, a^T and du^T, y^T --fp4q_gemm8--> the weights' gradients, in fp32
With --gated the layer is a = silu(gate y) * (up y): up is the joined weight of both, and in place
of the product and the activation stand fp4q_gated8 and fp4q_gated8_backward.  A token of a
serving step goes through the same weights as FP4 payloads: fp4q_gated4, fp4q_gemv4.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp4_communication_compression_amd as fp4q  # noqa: E402

EPS = 1e-6
E5M2 = torch.float8_e5m2


class Rank:
    """A rank's weight shards as 8-bit tiles, straight and transposed (made once per update)."""

    def __init__(self, up, down):
        self.up = fp4q.fp4q_quantize8(up, tiles=True, transposed=True)
        self.down = fp4q.fp4q_quantize8(down, tiles=True, transposed=True)

    def forward(self, norm):
        self.u = fp4q.fp4q_gemm8(norm.codes, norm.scales, self.up.codes, self.up.scales)
        a = self.u.clamp_min(0).square()
        self.a = fp4q.fp4q_quantize8(a, transposed=True)
        return fp4q.fp4q_gemm8(self.a.codes, self.a.scales, self.down.codes, self.down.scales)

    def backward(self, d, y_t):
        """This rank's part of dy; keeps the gradients of its weights."""
        da = fp4q.fp4q_gemm8(d.codes, d.scales, self.down.codes_t, self.down.scales_t)
        du = fp4q.fp4q_quantize8(2 * da * self.u.clamp_min(0), E5M2, transposed=True)
        self.ddown = fp4q.fp4q_gemm8(d.codes_t, d.scales_t, self.a.codes_t, self.a.scales_t, out_dtype=torch.float32)
        self.dup = fp4q.fp4q_gemm8(du.codes_t, du.scales_t, y_t.codes_t, y_t.scales_t, out_dtype=torch.float32)
        return fp4q.fp4q_gemm8(du.codes, du.scales, self.up.codes_t, self.up.scales_t)


class GatedRank(Rank):
    """A rank of a gated layer; up is the joined weight of the gate and the up projection."""

    def forward(self, norm):
        self.h = fp4q.fp4q_gated8(norm.codes, norm.scales, self.up.codes, self.up.scales, want_pre=True)
        a = fp4q.fp4q_quantize8(self.h.y)
        return fp4q.fp4q_gemm8(a.codes, a.scales, self.down.codes, self.down.scales)

    def backward(self, d, y_t):
        da = fp4q.fp4q_gemm8(d.codes, d.scales, self.down.codes_t, self.down.scales_t)
        g = fp4q.fp4q_gated8_backward(da, self.h.gate, self.h.up, want_y=True)
        self.ddown = fp4q.fp4q_gemm8(d.codes_t, d.scales_t, g.y_codes_t, g.y_scales_t, out_dtype=torch.float32)
        self.dup = fp4q.fp4q_gemm8(g.codes_t, g.scales_t, y_t.codes_t, y_t.scales_t, out_dtype=torch.float32)
        return fp4q.fp4q_gemm8(g.codes, g.scales, self.up.codes_t, self.up.scales_t)


class ServingRank:
    """A rank of a gated layer for single tokens: its weights as FP4 payloads, whose rows are
    whole blocks of 256 (the shard's inner width is padded with zeros)."""

    def __init__(self, up, down):
        n, flags = down.shape[1], fp4q.FP4Q_FLAG_NO_FWHT
        pad = torch.nn.functional.pad
        self.gate, self.up = (fp4q.fp4q_compress(pad(w, (0, 0, 0, -n % 256)), flags=flags) for w in (up[:n], up[-n:]))
        self.down = fp4q.fp4q_compress(pad(down, (0, -n % 256)), flags=flags)

    def forward(self, y):
        flags = fp4q.FP4Q_FLAG_NO_FWHT
        return fp4q.fp4q_gemv4(fp4q.fp4q_gated4(y, self.gate, self.up, flags=flags), self.down, flags=flags)


def exchange(parts, compress=True):
    """The AllReduce of the ranks' bf16 parts: every rank compresses its own and sums all."""
    if not compress:
        return torch.stack([p.float() for p in parts]).sum(dim=0).to(torch.bfloat16)
    return fp4q.fp4q_decompress_accumulate([fp4q.fp4q_compress(p) for p in parts], out_dtype=torch.bfloat16)


def layer(ranks, parts, residual, weight, d, compress=True):
    """Output, and the gradients of the summed input and the norm's weight."""
    x = exchange(parts, compress)
    norm = fp4q.fp4q_rmsnorm(x, weight, EPS, residual=residual, want_codes=True, want_rstd=True)
    out = exchange([r.forward(norm) for r in ranks], compress)
    qd = fp4q.fp4q_quantize8(d, E5M2, transposed=True)
    y_t = fp4q.fp4q_quantize8(norm.y, straight=False, transposed=True)
    dy = exchange([r.backward(qd, y_t) for r in ranks], compress)
    dx, dweight = fp4q.fp4q_rmsnorm_backward(dy, norm.h, weight, norm.rstd, dh=d)
    return out, dx, dweight


def activation(z, n, gated):
    """What stands between the two projections, n wide, in fp32."""
    return torch.nn.functional.silu(z[:, :n]) * z[:, -n:] if gated else z.clamp_min(0).square()


def reference(ups, downs, parts, residual, weight, d, gated=False):
    """The same layer in fp32, gradients by autograd."""
    x = sum(p.float() for p in parts).requires_grad_()
    ups, downs = ([w.float().requires_grad_() for w in ws] for ws in (ups, downs))
    w = weight.float().requires_grad_()
    h = x + residual.float()
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS) * w
    out = sum(activation(y @ u.t(), v.shape[1], gated) @ v.t() for u, v in zip(ups, downs))
    (out * d.float()).sum().add((h * d.float()).sum()).backward()
    return out.detach(), x.grad, w.grad, [u.grad for u in ups], [v.grad for v in downs]


def make(ranks, tokens, hidden, inner, device, seed=0, gated=False):
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    bf, n = torch.bfloat16, inner // ranks

    def up():
        if not gated:
            return rand(n, hidden)
        return torch.cat([rand(n, hidden), torch.zeros(-n % 128, hidden, device=device), rand(n, hidden)])

    ups = [(up() * hidden ** -0.5).to(bf) for _ in range(ranks)]
    downs = [(rand(hidden, inner // ranks) * inner ** -0.5).to(bf) for _ in range(ranks)]
    parts = [(rand(tokens, hidden) * ranks ** -0.5).to(bf) for _ in range(ranks)]
    weight = (1 + 0.1 * rand(hidden)).to(bf)
    return ups, downs, parts, rand(tokens, hidden).to(bf), weight, (0.1 * rand(tokens, hidden)).to(bf)


def off(a, b):
    return float((a.float() - b).norm() / b.norm())


def errors(ranks, tokens, hidden, inner, compress=True, device="cuda", gated=False):
    """Relative errors of the layer against fp32, by name."""
    ups, downs, parts, residual, weight, d = make(ranks, tokens, hidden, inner, device, gated=gated)
    shards = [(GatedRank if gated else Rank)(u, v) for u, v in zip(ups, downs)]
    out, dx, dw = layer(shards, parts, residual, weight, d, compress)
    want = reference(ups, downs, parts, residual, weight, d, gated)
    return {"output": off(out, want[0]), "dx": off(dx, want[1]), "dweight": off(dw, want[2]),
            "dup": max(off(r.dup, w) for r, w in zip(shards, want[3])),
            "ddown": max(off(r.ddown, w) for r, w in zip(shards, want[4]))}


def token_error(ranks, tokens, hidden, inner, device="cuda"):
    """Relative error of a serving step's tokens with 4-bit weights against fp32 with bf16 weights."""
    ups, downs, _, y, _, _ = make(ranks, tokens, hidden, inner, device, gated=True)
    out = exchange([ServingRank(u, v).forward(y) for u, v in zip(ups, downs)], compress=False)
    return off(out, sum(activation(y.float() @ u.float().t(), v.shape[1], True) @ v.float().t() for u, v in zip(ups, downs)))


def timed(call, count):
    """ms a call, among others."""
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    call()
    start.record()
    for _ in range(count):
        call()
    stop.record()
    torch.cuda.synchronize()
    return start.elapsed_time(stop) / count


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("ranks", 4), ("tokens", 2048), ("hidden", 4096), ("inner", 11008)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--gated", action="store_true")
    a = ap.parse_args()
    for compress in (False, True):
        e = errors(a.ranks, a.tokens, a.hidden, a.inner, compress, gated=a.gated)
        print("%-24s %s" % ("FP4 exchange" if compress else "uncompressed exchange",
                            "  ".join("%s %.3f" % kv for kv in e.items())))
    ups, downs, parts, residual, weight, d = make(a.ranks, a.tokens, a.hidden, a.inner, "cuda", gated=a.gated)
    shards = [(GatedRank if a.gated else Rank)(u, v) for u, v in zip(ups, downs)]
    print("forward and backward of all %d ranks: %.2f ms" % (
        a.ranks, timed(lambda: layer(shards, parts, residual, weight, d), 5)))
    if a.gated:
        rank, y = ServingRank(ups[0], downs[0]), residual[:1].contiguous()
        print("one token with 4-bit weights: error %.3f, one rank's layer %.1f us" % (
            token_error(a.ranks, 1, a.hidden, a.inner), 1e3 * timed(lambda: rank.forward(y), 200)))


if __name__ == "__main__":
    main()
