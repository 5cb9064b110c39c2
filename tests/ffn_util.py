"""64-bit references and inputs for the tests of the products with 4-bit weights and the layer
norm: plain numpy from the definitions of include/qz.h, no code of the library."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
FORMATS = {"mxfp4": 32, "nvfp4": 16, "int4": 128}


def bf16_round(v):
    """float64 -> the nearest bf16 (ties to even), as float64 (normal range)."""
    b = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def e4m3_value(b):
    b = np.asarray(b).astype(np.int64)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    return np.where(e > 0, np.ldexp(1 + m / 8, e - 7), m / 512)


def make_weight(rng, fmt, rows, cols, group=None, exact=False):
    """Random codes over all nibbles that the format uses, and scales.  exact: powers of two
    near 1, so that products with small integers sum without rounding."""
    group = group or FORMATS[fmt]
    nib = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    if fmt == "int4":
        nib = np.where(nib == 8, 0, nib).astype(np.uint8)
        val = np.where(nib >= 8, nib.astype(np.int64) - 16, nib).astype(np.float64)
    else:
        val = np.where(nib >= 8, -1.0, 1.0) * E2M1[nib & 7]
    shape = (rows, cols // group)
    ts = np.float32(1.0)
    if fmt == "int4":
        sc = np.ldexp(1.0, rng.integers(-2, 2, shape)) if exact else rng.uniform(0.001, 0.02, shape)
        sc = sc.astype(np.float32)
        k = sc.astype(np.float64)
    elif fmt == "mxfp4":
        sc = (rng.integers(-2, 2, shape) if exact else rng.integers(-9, 1, shape)) + 127
        k = np.ldexp(1.0, sc - 127)
        sc = sc.astype(np.uint8)
    else:
        sc = (np.int64(7) + rng.integers(-2, 2, shape)) << 3 if exact else rng.integers(0, 0x7F, shape)
        k = e4m3_value(sc)
        sc = sc.astype(np.uint8)
        ts = np.float32(0.25 if exact else rng.uniform(1e-4, 1e-3))
        k = k * np.float64(ts)
    codes = (nib[:, 0::2] | (nib[:, 1::2] << 4)).astype(np.uint8)
    return dict(fmt=fmt, group=group, rows=rows, cols=cols, codes=codes, scales=sc, ts=ts,
                elements=val, values=val * np.repeat(k, group, axis=1))


def handle(w):
    import torch

    import precision_quantization_gb300 as qz
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    q = qz.Quantized(t(w["codes"]), t(w["scales"]), t(np.array([w["ts"]], np.float32)),
                     qz.FORMATS[w["fmt"]], qz.QZ_GRAN_BLOCK, qz.QZ_SCALE_UP, w["rows"], w["cols"],
                     w["group"])
    return qz.Weight(q)


def activations(rng, tokens, cols, exact=False, scale=1.0):
    if exact:
        return rng.integers(-4, 5, (tokens, cols)).astype(np.float64)
    return bf16_round(rng.normal(0, scale, (tokens, cols)))


def bf16_cuda(a, pad=0, lead=0):
    """A float64 array of bf16 values as a CUDA tensor; a view with `pad` unused columns after
    and `lead` before each row (filled with NaN, which no call may read into a result)."""
    import torch
    t = torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16)
    if pad or lead:
        big = torch.full((a.shape[0], lead + a.shape[1] + pad), float("nan"), dtype=torch.bfloat16)
        big[:, lead:lead + a.shape[1]] = t
        return big.cuda()[:, lead:lead + a.shape[1]]
    return t.cuda()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def act(a, kind):
    """The activation and its derivative."""
    with np.errstate(over="ignore"):
        if kind == "silu":
            p = 1 / (1 + np.exp(-a))
            return a * p, p + a * p * (1 - p)
        c = np.sqrt(2 / np.pi)
        th = np.tanh(c * (a + 0.044715 * a ** 3))
        return 0.5 * a * (1 + th), 0.5 * (1 + th) + 0.5 * a * (1 - th ** 2) * c * (1 + 3 * 0.044715 * a ** 2)


def sum_bound(k, terms):
    """How far an fp32 sum of k products may be from the exact one, `terms` = sum |products|.
    34 units of 2^-24 per 16 terms cover a tensor-core step (16 exact products aligned to the
    largest addend and truncated to 24 bits, two more for the normalisation: qz_quant_dot
    derives it) and any order of separately rounded adds (16 per 16 terms); 2^-17 covers an INT4
    weight held as the sum of two bf16 values (each keeps 8 bits); 64 units the joins, the tensor
    scale and the weight's own rounding."""
    return (34 * (k / 16 + 1) + 64) * 2.0 ** -24 * terms + 2.0 ** -17 * terms


def bf16_bound(v):
    """Half a unit in the last place of bf16: 8 significant bits, so 2^-8 of the value at the start
    of a binade; one per cent more for a result that the sum's own bound moves across one."""
    return 2.0 ** -8 * np.abs(v) * 1.01 + 1e-38


def assert_within(got, want, bound, what=""):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3],
                           np.broadcast_to(bound, got.shape)[bad][:3])
