"""The feed-forward half of a transformer layer on 4-bit weights:

    n = layer_norm(x),  h = silu(n gate^T) * (n up^T),  y = x + h down^T

quantizes the three weights, runs a prompt forward and backward (the codes are frozen: the
gradients are those of x and of the norm's weight and bias), then decodes one token, and
compares everything with the same block in fp32 on the dequantized weights.

    python examples/feed_forward_block.py [--format mxfp4|nvfp4|int4] [--tokens N] [--hidden D] [--inner F]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import precision_quantization_gb300 as qz


class FeedForward:
    """The block's weights: three quantized matrices and the norm's parameters."""

    def __init__(self, gate, up, down, fmt: str, norm_weight, norm_bias):
        self.gate, self.up, self.down = (qz.Weight(qz.quantize(w, fmt)[0]) for w in (gate, up, down))
        self.norm_weight, self.norm_bias = norm_weight, norm_bias

    def forward(self, x):
        """y and what the backward pass needs."""
        n, mean, rstd = qz.layer_norm(x, self.norm_weight, self.norm_bias)
        h, g, u = qz.gated_ffn(n, self.gate, self.up, save=True)
        return x + qz.linear(h, self.down), (x, mean, rstd, g, u)

    def backward(self, dy, kept):
        """dx and the gradients of the norm's weight and bias."""
        x, mean, rstd, g, u = kept
        dh = qz.linear_backward(dy, self.down)
        dn, _, _ = qz.gated_ffn_backward(dh, g, u, self.gate, self.up)
        dx, dweight, dbias = qz.layer_norm_backward(dn, x, mean, rstd, self.norm_weight)
        return dx + dy, dweight, dbias

    def decode(self, x):
        """One token: nothing is kept."""
        n, _, _ = qz.layer_norm(x, self.norm_weight, self.norm_bias)
        return x + qz.linear(qz.gated_ffn(n, self.gate, self.up), self.down)


def reference(block: FeedForward, x):
    """The block in fp32 on the dequantized weights, through autograd."""
    gate, up, down = (qz.dequantize(w.q, torch.float32) for w in (block.gate, block.up, block.down))
    n = torch.nn.functional.layer_norm(x, x.shape[-1:], block.norm_weight, block.norm_bias)
    return x + (torch.nn.functional.silu(n @ gate.T) * (n @ up.T)) @ down.T


def relative(a, b) -> float:
    return float((a.float() - b).norm() / b.norm())


def run(fmt: str = "nvfp4", tokens: int = 300, hidden: int = 1024, inner: int = 2816, seed: int = 0) -> dict:
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    gate, up, down = ((normal(*s) * s[1] ** -0.5).to(torch.bfloat16) for s in ((inner, hidden), (inner, hidden), (hidden, inner)))
    block = FeedForward(gate, up, down, fmt, 1 + 0.1 * normal(hidden), 0.1 * normal(hidden))
    x, dy = normal(tokens, hidden).to(torch.bfloat16), normal(tokens, hidden).to(torch.bfloat16)
    y, kept = block.forward(x)
    dx, dweight, dbias = block.backward(dy, kept)
    token = block.decode(x[-1:])

    xr = x.float().requires_grad_()
    block.norm_weight.requires_grad_()
    block.norm_bias.requires_grad_()
    want = reference(block, xr)
    want.backward(dy.float())
    errors = {"y": relative(y, want.detach()), "dx": relative(dx, xr.grad),
              "dweight": relative(dweight, block.norm_weight.grad), "dbias": relative(dbias, block.norm_bias.grad),
              "decoded token": relative(token, want.detach()[-1:])}
    return errors


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--format", choices=("mxfp4", "nvfp4", "int4"), default="nvfp4")
    ap.add_argument("--tokens", type=int, default=300)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=2816)
    a = ap.parse_args()
    for name, e in run(a.format, a.tokens, a.hidden, a.inner).items():
        print(f"{name:14s} relative difference from fp32 on the same weights: {e:.2e}")


if __name__ == "__main__":
    main()
