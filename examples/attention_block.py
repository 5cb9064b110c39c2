"""The attention half of a transformer layer on 4-bit weights and an 8-bit key-value cache:

    n = layer_norm(x),  (q, k, v) = n Wqkv^T,  append k and v to the cache (q and k rotated by position),
    o = attention(q, cache),  y = x + o Wo^T

runs prompts of several sequences and then decodes tokens, and compares each stage with fp32 on the
same inputs: the projections on the dequantized weights, the attention on the values that the cache
holds.

    python examples/attention_block.py [--format mxfp4|nvfp4|int4] [--cache int8|e4m3|e5m2] [--heads H] [--kv-heads K] [--dim D]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import precision_quantization_gb300 as qz


class Attention:
    """The block's weights, its cache and its rotation; pages are handed out in order."""

    def __init__(self, wqkv, wo, fmt: str, heads: int, kv_heads: int, dim: int, sequences: int, positions: int, cache: str = "e4m3",
                 page: int = 64, block: int = 32):
        self.qkv, self.out = (qz.Weight(qz.quantize(w, fmt)[0]) for w in (wqkv, wo))
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        each = -(-positions // page)
        self.cache = qz.KVCache.alloc(cache, sequences * each, kv_heads, page, dim, block)
        self.table = torch.arange(sequences * each, dtype=torch.int32, device="cuda").view(sequences, each)
        self.lengths = torch.zeros(sequences, dtype=torch.int32, device="cuda")
        self.rotary = qz.RotaryTable.make(positions, qz.rotary_turns(dim // 2))

    def forward(self, x, starts=None):
        """x [tokens, hidden]: the new tokens of every sequence, one each, or starts[i] .. starts[i + 1] - 1."""
        self.lengths += 1 if starts is None else starts.diff()
        n, _, _ = qz.layer_norm(x)
        qkv = qz.linear(n, self.qkv).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)  # slices: nothing is copied
        q = qz.cache_append(self.cache, k, v, self.table, self.lengths, starts, rotary=self.rotary, q=q)
        o = qz.cache_attention(q, self.cache, self.table, self.lengths, starts)
        return x + qz.linear(o.view(x.shape[0], -1), self.out), (q, o)


def cache_values(block: Attention, which: str):
    """What the cache holds, fp32 [sequences, kv_heads, positions, dim]."""
    c = block.cache
    codes, scales = (c.k_codes, c.k_scales) if which == "k" else (c.v_codes, c.v_scales)
    view = {qz.QZ_INT8: torch.int8, qz.QZ_FP8_E4M3: torch.float8_e4m3fn, qz.QZ_FP8_E5M2: torch.float8_e5m2}[c.fmt]
    x = codes.view(view).float().view(c.pages, c.kv_heads, -1, c.block, c.dim) * scales[..., None, None]
    x = x.view(c.pages, c.kv_heads, c.page, c.dim)[block.table.long()]          # [sequences, pages, heads, page, dim]
    return x.transpose(1, 2).flatten(2, 3)


def reference(block: Attention, q, starts):
    """The attention in fp32 on the cache's values."""
    k, v = cache_values(block, "k"), cache_values(block, "v")
    out, group = torch.empty(q.shape, device="cuda"), block.heads // block.kv_heads
    for s, length in enumerate(block.lengths.tolist()):
        r0, r1 = starts[s], starts[s + 1]
        x = q[r0:r1].float().transpose(0, 1)                                     # [heads, tokens, dim]
        ks, vs = (t[s, :, :length].repeat_interleave(group, 0) for t in (k, v))
        score = x @ ks.transpose(-1, -2) * block.dim ** -0.5
        last = torch.arange(length - (r1 - r0), length, device="cuda")
        score.masked_fill_(torch.arange(length, device="cuda") > last[:, None], -torch.inf)
        out[r0:r1] = (score.softmax(-1) @ vs).transpose(0, 1)
    return out


def relative(a, b) -> float:
    return float((a.float() - b).norm() / b.norm())


def run(fmt: str = "nvfp4", cache: str = "e4m3", heads: int = 16, kv_heads: int = 4, dim: int = 64, prompts=(200, 77, 1), steps: int = 3,
        seed: int = 0) -> dict:
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    hidden = heads * dim
    wqkv, wo = ((normal(*s) * s[1] ** -0.5).to(torch.bfloat16) for s in (((heads + 2 * kv_heads) * dim, hidden), (hidden, hidden)))
    block = Attention(wqkv, wo, fmt, heads, kv_heads, dim, len(prompts), max(prompts) + steps, cache)
    out = qz.dequantize(block.out.q, torch.float32)
    errors = {}

    def step(name, x, starts):
        y, (q, o) = block.forward(x, None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda"))
        rows = starts or list(range(len(prompts) + 1))
        errors["attention, " + name] = max(errors.get("attention, " + name, 0.0), relative(o, reference(block, q, rows)))
        errors["y, " + name] = max(errors.get("y, " + name, 0.0), relative(y, x.float() + o.float().flatten(1) @ out.T))

    starts = [sum(prompts[:i]) for i in range(len(prompts) + 1)]
    step("prompts", normal(starts[-1], hidden).to(torch.bfloat16), starts)
    for _ in range(steps):
        step("decoded tokens", normal(len(prompts), hidden).to(torch.bfloat16), None)
    return errors


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--format", choices=("mxfp4", "nvfp4", "int4"), default="nvfp4")
    ap.add_argument("--cache", choices=("int8", "e4m3", "e5m2"), default="e4m3")
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv-heads", type=int, default=4)
    ap.add_argument("--dim", type=int, default=64)
    a = ap.parse_args()
    for name, e in run(a.format, a.cache, a.heads, a.kv_heads, a.dim).items():
        print(f"{name:28s} relative difference from fp32 on the same inputs: {e:.2e}")


if __name__ == "__main__":
    main()
