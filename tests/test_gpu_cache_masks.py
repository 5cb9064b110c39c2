"""Attention to the 8-bit cache where blocks that a row does not see hold values out of all proportion: the row keeps the
accuracy that the blocks it sees allow."""
import numpy as np
import pytest

import cache_util as U
from test_gpu_cache import check, gpu, on_gpu, qz, sequences  # noqa: F401

pytestmark = pytest.mark.gpu

MASKED = [  # lengths, new tokens, page, block, heads, kv, dim, window, positions whose block is spoiled (of each sequence)
    ([146, 50], [3, 2], 64, 16, 8, 2, 64, 0, [144, 48]),          # a block that only the later tokens see, and its neighbours' step
    ([146, 50], [3, 2], 64, 16, 8, 2, 128, 0, [144, 48]),
    ([146, 50], [3, 2], 32, 16, 8, 2, 256, 0, [144, 48]),
    ([146, 150], [3, 3], 64, 16, 32, 4, 128, 0, [144, 144]),      # 24 rows
    ([200, 1000], [2, 2], 64, 16, 8, 2, 64, 152, [47, 848]),      # before a window: the first token sees its last position
    ([1000, 1900], [1, 1], 64, 16, 8, 2, 128, 903, [96, 992]),    # or none does
    ([1000, 900], [4, 3], 16, 16, 32, 4, 64, 903, [94, 0]),
    ([4000, 900], [2, 2], 64, 16, 4, 1, 128, 3000, [999, 0]),     # cut into shares
    ([200], [90], 64, 16, 4, 2, 64, 0, [176]),                    # prompts
    ([300, 140], [150, 77], 32, 16, 8, 2, 128, 0, [240, 112]),
    ([333, 200], [200, 64], 32, 32, 4, 2, 64, 100, [64, 64]),
    ([1100, 40], [150, 40], 32, 16, 4, 2, 96, 700, [320, 16]),    # cut along the keys
]


def wanted(q, host, table, lengths, starts, scale, window):
    """U.attention's, with what small weights lose by the largest scale of values that the row sees (a weight times its
    scale is off by 2^-25 2^-11 of a unit up to eight times that scale: 2^-33 of it for each code; 2^-29 allows for a
    unit that is 2^4 above), every weight 1 at most and their sum 1 at least."""
    out, lse, mag, err, floor = U.attention(q, host, table, lengths, starts, scale, window)
    group = q.shape[1] // host.heads
    for s, length in enumerate(lengths):
        n = starts[s + 1] - starts[s]
        at = np.arange(length)
        vs = np.stack([host.scales[1][table[s, j // host.page], :, j % host.page // host.block] for j in at]).astype(np.float64)
        for i in range(n):
            pos = length - n + i
            seen = (at <= pos) & (at > (pos - window if window else -1))
            for h in range(q.shape[1]):
                floor[starts[s] + i, h] = 2.0 ** -29 * vs[seen, h // group].max() * U.QMAX[host.fmt] * seen.sum() + 2.0 ** -126
    return out, lse, mag, err, floor


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 96])
@pytest.mark.parametrize("case", range(len(MASKED)))
def test_large_values_that_a_row_does_not_see(qz, fmt, size, case):  # noqa: F811
    lengths, new, page, block, heads, kv, dim, window, spoiled = MASKED[case]
    rng = np.random.default_rng(case)
    seqs, tokens = len(lengths), sum(new)
    each = -(-max(lengths) // page)
    host = U.Cache(rng, fmt, seqs * each + 1, kv, page, dim, block)
    table = sequences(rng, seqs, each, host.pages)
    for s in range(seqs):
        host.fill(rng, table[s], lengths[s])
        if spoiled[s]:
            host.scales[1][table[s, spoiled[s] // page], :, spoiled[s] % page // block] *= np.float32(size)
    q = U.bf16((2 * rng.standard_normal((tokens, heads, dim))).astype(np.float32))
    starts, scale = np.concatenate(([0], np.cumsum(new))).astype(np.int32), 0.02
    out, lse = qz.cache_attention(gpu(q).bfloat16(), on_gpu(qz, host), gpu(table), gpu(np.array(lengths, np.int32)), gpu(starts),
                                  scale=scale, window=window or None, lse=True)
    check(out, lse, wanted(q.astype(np.float64), host, table, lengths, starts, scale, window))


NONFINITE = {"e4m3": [0x7F, 0xFF], "e5m2": [0x7C, 0x7F, 0xFC, 0xFD]}


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("which", ["keys", "values"])
@pytest.mark.parametrize("case", range(len(MASKED)))
def test_codes_that_are_no_numbers_spoil_the_rows_that_see_them(qz, fmt, which, case):  # noqa: F811
    """NaN and Inf codes just before the first token's window, at its first position and at the last token's own."""
    lengths, new, page, block, heads, kv, dim, window, _ = MASKED[case]
    rng = np.random.default_rng(50 + case)
    seqs, tokens = len(lengths), sum(new)
    each = -(-max(lengths) // page)
    host = U.Cache(rng, fmt, seqs * each + 1, kv, page, dim, block)
    table = sequences(rng, seqs, each, host.pages)
    for s in range(seqs):
        host.fill(rng, table[s], lengths[s])
    q = U.bf16((2 * rng.standard_normal((tokens, heads, dim))).astype(np.float32))
    starts, scale = np.concatenate(([0], np.cumsum(new))).astype(np.int32), dim ** -0.5
    out, lse, *rest = U.attention(q.astype(np.float64), host, table, lengths, starts, scale, window)
    sees = np.zeros(tokens, bool)
    for s, length in enumerate(lengths):
        at = np.arange(length - new[s], length)
        first = np.maximum(at - window + 1, 0) if window else np.zeros(new[s], int)
        for p in {int(first[0]) - 1, int(first[0]) if first[-1] > first[0] else -1, length - 1 if new[s] > 1 else -1} - {-1}:
            codes = host.codes[which == "values"][table[s, p // page], :, p % page]
            codes[:, rng.integers(0, dim)] = 0x7F    # a NaN of either format
            if not ((p <= at) & (p >= first)).any():
                codes[:] = rng.choice(NONFINITE[fmt], codes.shape)
            sees[starts[s]:starts[s + 1]] |= (p <= at) & (p >= first)
    got, logs = qz.cache_attention(gpu(q).bfloat16(), on_gpu(qz, host), gpu(table), gpu(np.array(lengths, np.int32)), gpu(starts),
                                   scale=scale, window=window or None, lse=True)
    keep = ~sees
    assert keep.any() or sees.all()
    if keep.any():
        check(got[gpu(keep)], logs[gpu(keep)], (out[keep], lse[keep], *(r[keep] for r in rest)))
    assert (~np.isfinite(got[gpu(sees)].double().cpu().numpy())).any(-1).all()
