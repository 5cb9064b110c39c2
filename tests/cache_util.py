"""References and inputs for the tests of the rotation by positions, the paged 8-bit cache and the
attention that reads it: plain numpy from the definitions of include/qz.h, no code of the library."""
from __future__ import annotations

import numpy as np

QMAX = {"int8": 127.0, "e4m3": 448.0, "e5m2": 57344.0}
F32 = np.float32


def code_values(codes, fmt):
    """What the codes (uint8) stand for, float64; E4M3 0x7F and E5M2's last codes are NaN and Inf."""
    c = np.asarray(codes).astype(np.int64)
    if fmt == "int8":
        return np.where(c > 127, c - 256, c).astype(np.float64)
    m, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    e, f = (c & 127) >> m, (c & ((1 << m) - 1)) / (1 << m)
    v = np.where(e > 0, (1 + f) * 2.0 ** (e - bias), f * 2.0 ** (1 - bias))
    if fmt == "e4m3":
        v = np.where((c & 127) == 127, np.nan, v)
    else:
        v = np.where(e == 31, np.where(f == 0, np.inf, np.nan), v)
    return np.where(c > 127, -v, v)


def nearest_codes(v, fmt):
    """The codes nearest to fp32 values, ties to even, saturating."""
    v = np.asarray(v, F32)
    if fmt == "int8":
        return np.clip(np.rint(v), -127, 127).astype(np.int8).view(np.uint8)
    m, least, bias = (3, -6, 7) if fmt == "e4m3" else (2, -14, 15)
    a = np.minimum(np.abs(v).astype(np.float64), QMAX[fmt])
    e = np.maximum(np.frexp(a)[1] - 1, least)
    n = np.rint(a / 2.0 ** (e - m)).astype(np.int64)   # a = n 2^(e - m), n up to 2^(m + 1)
    e, n = np.where(n == 2 << m, e + 1, e), np.where(n == 2 << m, 1 << m, n)
    code = np.where(n >= 1 << m, ((e + bias) << m) + n - (1 << m), n)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def rotated(x, cos, sin, interleaved, back=False):
    """x fp32 [..., dim] with cos, sin fp32 [..., pairs]: fp32, each product and sum rounded."""
    pairs = cos.shape[-1]
    y = np.array(x, F32)
    a, b = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if interleaved else (slice(0, pairs), slice(pairs, 2 * pairs))
    x1, x2, s = y[..., a].copy(), y[..., b].copy(), -sin if back else sin
    y[..., a] = x1 * cos - x2 * s
    y[..., b] = x2 * cos + x1 * s
    return y


def bf16(v):
    """fp32 -> the nearest bf16 (ties to even), as fp32; NaN stays NaN."""
    v = np.asarray(v, F32)
    b = v.view(np.uint32).astype(np.uint64)
    r = (((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)).view(F32)
    return np.where(np.isnan(v), v, r)


class Cache:
    """A cache on the host.  Slots that no test fills hold what uninitialised memory may."""

    def __init__(self, rng, fmt, pages, heads, page, dim, block, junk=True):
        self.fmt, self.page, self.dim, self.block, self.heads, self.pages = fmt, page, dim, block, heads, pages
        shape = (pages, heads, page, dim)
        self.codes = [rng.integers(0, 256, shape).astype(np.uint8) if junk else np.zeros(shape, np.uint8) for _ in range(2)]
        self.scales = [np.full((pages, heads, page // block), np.nan if junk else 0.0, F32) for _ in range(2)]

    def fill(self, rng, pages_of, length, spread=1.0):
        """Ordinary codes and scales for the first `length` positions of a sequence."""
        for c, s in zip(self.codes, self.scales):
            for j in range(0, length, self.block):
                p = pages_of[j // self.page]
                if p < 0:
                    continue
                at = j % self.page
                n = min(self.block, length - j)
                x = rng.standard_normal((self.heads, n, self.dim)) * np.exp(spread * rng.standard_normal((self.heads, 1, 1)))
                scale = (np.abs(x).max((1, 2)) / QMAX[self.fmt]).astype(F32)
                s[p, :, at // self.block] = scale
                c[p, :, at:at + n] = nearest_codes((x / scale[:, None, None]).astype(F32), self.fmt)

    def gather(self, which, pages_of, length):
        """Values [heads, length, dim] in float64 and which positions have a page."""
        out, there = np.zeros((self.heads, length, self.dim)), np.zeros(length, bool)
        for j in range(length):
            p = pages_of[j // self.page] if j // self.page < len(pages_of) else -1
            if not 0 <= p < self.pages:
                continue
            there[j] = True
            at = j % self.page
            out[:, j] = code_values(self.codes[which][p, :, at], self.fmt) * self.scales[which][p, :, at // self.block].astype(np.float64)[:, None]
        return out, there

    def append(self, k, v, table, lengths, starts, cos, sin, interleaved):
        """include/qz.h's append, to the bit: k, v fp32 [tokens, heads, dim]."""
        for s, length in enumerate(lengths):
            row, n = starts[s], starts[s + 1] - starts[s]
            p0 = length - n
            first = max(p0, 0)
            end = min(length, len(table[s]) * self.page, *([cos.shape[0]] if cos is not None else []))
            for b0 in range(first // self.block * self.block, end, self.block):
                page = table[s][b0 // self.page]
                if not 0 <= page < self.pages:
                    continue
                lo, hi, at = max(first, b0), min(end, b0 + self.block), b0 % self.page
                if lo >= hi:
                    continue
                rows = row + np.arange(lo, hi) - p0
                for which, x in enumerate((k[rows], v[rows])):
                    if which == 0 and cos is not None:
                        x = rotated(x, cos[lo:hi, None], sin[lo:hi, None], interleaved)
                    codes, scales = self.codes[which][page], self.scales[which][page]
                    for h in range(self.heads):
                        old = scales[h, at // self.block] if lo > b0 else F32(0)
                        a = F32(np.abs(x[:, h]).max())  # (NaN stays NaN)
                        now = np.maximum(F32(a / F32(QMAX[self.fmt])), old)
                        scales[h, at // self.block] = now
                        held = codes[h, at:at + lo - b0]
                        bad = not np.isfinite(now)
                        if bad:
                            held[:] = 0
                        elif now > old and lo > b0:
                            held[:] = nearest_codes(code_values(held, self.fmt).astype(F32) * F32(old / now), self.fmt)
                        new = 0 if bad or now == 0 else nearest_codes(x[:, h] / now, self.fmt)
                        codes[h, at + lo - b0:at + hi - b0] = new


def attention(q, cache: Cache, table, lengths, starts, scale, window=0):
    """(out, lse, magnitude, exponent error, floor) in float64: q [tokens, heads, dim] (the values the
    library gets), magnitude = sum p |v|, the bound on the error of a score in units of log (fp32
    tensor-core sums, 34 x 2^-24 of the terms' magnitudes for each 16: one step c + 16 exact products cut
    to 24 bits and normalised), and what is lost where a weight p x scale is small: as f16 times 2^-11 of
    the unit it is off by 2^-25 2^-11 of the unit, a power of two up to eight times the sequence's largest
    scale of values, against a p of the largest score of 2^-4 at least (the maximum is followed that far
    behind), so each code of a visible position contributes up to 2^-29 of that scale (and no less than
    fp32's smallest normal number, 2^-126)."""
    tokens, heads, dim = q.shape
    group = heads // cache.heads
    out, lse = np.full((tokens, heads, dim), np.nan), np.full((tokens, heads), np.nan)
    mag, floor, err = np.zeros((tokens, heads, dim)), np.zeros((tokens, heads, dim)), np.zeros((tokens, heads))
    for s, length in enumerate(lengths):
        row, n = starts[s], starts[s + 1] - starts[s]
        length = max(length, 0)
        held = min(length, len(table[s]) * cache.page)
        k, there = cache.gather(0, table[s], held)
        v, _ = cache.gather(1, table[s], held)
        unit = np.zeros(cache.heads)
        for p in table[s][:-(-held // cache.page)]:
            if 0 <= p < cache.pages:
                with np.errstate(all="ignore"):
                    unit = np.fmax(unit, np.nanmax(np.append(cache.scales[1][p], np.zeros((cache.heads, 1)), 1), 1))
        for i in range(n):
            pos = length - n + i
            seen = there & (np.arange(held) <= pos)
            if window:
                seen &= np.arange(held) > pos - window
            for h in range(heads):
                kk, vv = k[h // group][seen], v[h // group][seen]
                if not len(kk):
                    out[row + i, h], lse[row + i, h] = 0.0, -np.inf
                    continue
                with np.errstate(all="ignore"):
                    x = kk @ q[row + i, h] * scale
                    top = x.max()
                    p = np.exp(x - top)
                    out[row + i, h], lse[row + i, h] = p @ vv / p.sum(), top + np.log(p.sum())
                    mag[row + i, h] = p @ np.abs(vv) / p.sum()
                    floor[row + i, h] = 2.0 ** -29 * unit[h // group] * QMAX[cache.fmt] * len(vv) / p.sum() + 2.0 ** -126
                    err[row + i, h] = 34 * -(-dim // 16) * 2.0 ** -24 * scale * (np.abs(kk) @ np.abs(q[row + i, h])).max()
    return out, lse, mag, err, floor


def attention_tolerance(out, lse, mag, err, floor):
    """Per element: the bf16 rounding of the result (2^-8), the weights' rounding to f16 (2^-11), the
    scores' error in numerator and denominator, exponentials and fp32 sums (2^-16 covers 2^-22 of an
    exponential and a few hundred roundings of partial sums).  lse: the scores' error, and fp32 (2^-20
    relative to its own size and that of the logarithms it is made of)."""
    rest = 2.0 ** -11 + 2 * err[..., None] + 2.0 ** -16
    with np.errstate(all="ignore"):
        return 2.0 ** -8 * np.abs(out) + rest * mag * 1.01 + floor, err + 2.0 ** -16 + 2.0 ** -20 * np.abs(np.where(np.isinf(lse), 0, lse))
