"""One tensor-parallel MLP layer, forward and backward, with the ranks of one group emulated
in turn on one GPU: what leaves a rank is FP4-compressed, what a rank computes runs on 8-bit
operands with a scale per 128.

    python examples/tp_layer.py [--ranks 4] [--tokens 2048] [--hidden 4096] [--inner 11008]

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


def reference(ups, downs, parts, residual, weight, d):
    """The same layer in fp32, gradients by autograd."""
    x = sum(p.float() for p in parts).requires_grad_()
    ups, downs = ([w.float().requires_grad_() for w in ws] for ws in (ups, downs))
    w = weight.float().requires_grad_()
    h = x + residual.float()
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS) * w
    out = sum((y @ u.t()).clamp_min(0).square() @ v.t() for u, v in zip(ups, downs))
    (out * d.float()).sum().add((h * d.float()).sum()).backward()
    return out.detach(), x.grad, w.grad, [u.grad for u in ups], [v.grad for v in downs]


def make(ranks, tokens, hidden, inner, device, seed=0):
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    bf = torch.bfloat16
    ups = [(rand(inner // ranks, hidden) * hidden ** -0.5).to(bf) for _ in range(ranks)]
    downs = [(rand(hidden, inner // ranks) * inner ** -0.5).to(bf) for _ in range(ranks)]
    parts = [(rand(tokens, hidden) * ranks ** -0.5).to(bf) for _ in range(ranks)]
    weight = (1 + 0.1 * rand(hidden)).to(bf)
    return ups, downs, parts, rand(tokens, hidden).to(bf), weight, (0.1 * rand(tokens, hidden)).to(bf)


def errors(ranks, tokens, hidden, inner, compress=True, device="cuda"):
    """Relative errors of the layer against fp32, by name."""
    ups, downs, parts, residual, weight, d = make(ranks, tokens, hidden, inner, device)
    shards = [Rank(u, v) for u, v in zip(ups, downs)]
    out, dx, dw = layer(shards, parts, residual, weight, d, compress)
    want = reference(ups, downs, parts, residual, weight, d)
    off = lambda a, b: float((a.float() - b).norm() / b.norm())  # noqa: E731
    return {"output": off(out, want[0]), "dx": off(dx, want[1]), "dweight": off(dw, want[2]),
            "dup": max(off(r.dup, w) for r, w in zip(shards, want[3])),
            "ddown": max(off(r.ddown, w) for r, w in zip(shards, want[4]))}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("ranks", 4), ("tokens", 2048), ("hidden", 4096), ("inner", 11008)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    for compress in (False, True):
        e = errors(a.ranks, a.tokens, a.hidden, a.inner, compress)
        print("%-24s %s" % ("FP4 exchange" if compress else "uncompressed exchange",
                            "  ".join("%s %.3f" % kv for kv in e.items())))
    ups, downs, parts, residual, weight, d = make(a.ranks, a.tokens, a.hidden, a.inner, "cuda")
    shards = [Rank(u, v) for u, v in zip(ups, downs)]
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    layer(shards, parts, residual, weight, d)
    start.record()
    for _ in range(5):
        layer(shards, parts, residual, weight, d)
    stop.record()
    torch.cuda.synchronize()
    print("forward and backward of all %d ranks: %.2f ms" % (a.ranks, start.elapsed_time(stop) / 5))


if __name__ == "__main__":
    main()
