"""The append's and the attention's launch forms that the sizes of test_gpu_cache.py do not reach: queries in a launch of
their own (256 tokens and more), blocks of four pieces a thread, more sequences than a CTA has threads."""
import numpy as np
import pytest

import cache_util as U
from test_gpu_cache import check, gpu, on_gpu, qz, same_bits, same_cache, sequences, table_of  # noqa: F401

pytestmark = pytest.mark.gpu


def appended(qz, fmt, dtype, lengths, new, page, block, heads, kv, dim, pairs, interleaved, form, seed, tail=0):  # noqa: F811
    """An append with rotated queries against numpy, to the bit; `tail` rows behind the last sequence stay as they are."""
    import torch
    rng = np.random.default_rng(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    seqs, tokens = len(lengths), sum(new)
    pages = [-(-n // page) for n in lengths]
    host = U.Cache(rng, fmt, sum(pages) + 2, kv, page, dim, block)
    order = rng.permutation(host.pages)
    table = np.full((seqs, max(pages)), -1, np.int32)
    for s, n in enumerate(pages):
        table[s, :n] = order[sum(pages[:s]):sum(pages[:s]) + n]
        host.fill(rng, table[s], max(lengths[s] - new[s], 0))
    rnd = lambda *s: (lambda v: U.bf16(v) if dtype == "bf16" else v)((1.5 * rng.standard_normal(s)).astype(np.float32))  # noqa: E731
    k, v, q = rnd(tokens + tail, kv, dim), rnd(tokens + tail, kv, dim), rnd(tokens + tail, heads, dim)
    cos, sin = table_of(max(lengths), pairs)
    starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    tk, tv, tq = (gpu(a, dt) for a in (k, v, q))
    if form == "slice":
        fused = torch.cat((tq, tk, tv), 1)
        tq, tk, tv = fused[:, :heads], fused[:, heads:heads + kv], fused[:, heads + kv:]
    elif form == "odd":
        shift = lambda t: torch.cat((t.new_zeros(1), t.reshape(-1)))[1:].view(t.shape)  # noqa: E731
        tq, tk, tv = shift(tq), shift(tk), shift(tv)
    cache, rot = on_gpu(qz, host), qz.RotaryTable(gpu(cos), gpu(sin), interleaved)
    out = torch.full(tq.shape, 7.0, dtype=dt, device="cuda")
    args = (cache, tk, tv, gpu(table), gpu(np.array(lengths, np.int32)), gpu(starts))
    assert qz.cache_append(*args, rotary=rot, q=tq, out=out) is out
    host.append(k, v, table, lengths, starts, cos, sin, interleaved)
    same_cache(cache, host)
    at = np.concatenate([np.arange(n - m, n) for n, m in zip(lengths, new)]).astype(int)
    want = U.rotated(q[:tokens], cos[at][:, None], sin[at][:, None], interleaved)
    assert same_bits(out[:tokens].float().cpu().numpy(), U.bf16(want) if dtype == "bf16" else want)
    assert (out[tokens:] == 7).all()
    mine = tq.clone()   # in place: the same bits, and the rest of the rows as it was
    qz.cache_append(*args, rotary=rot, q=mine, out=mine)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(mine[:tokens].view(bits), out[:tokens].view(bits)) and torch.equal(mine[tokens:], tq[tokens:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", ["dense", "slice", "odd"])
@pytest.mark.parametrize("interleaved,heads,kv,dim,pairs", [(False, 8, 2, 64, 32), (True, 5, 1, 128, 64), (False, 4, 2, 80, 9), (True, 70, 2, 32, 8)])
@pytest.mark.parametrize("lengths,new", [([300, 7], [256, 0]), ([150, 260, 90, 40], [111, 200, 90, 1])])
def test_queries_in_a_launch_of_their_own(qz, dtype, form, interleaved, heads, kv, dim, pairs, lengths, new):  # noqa: F811
    appended(qz, "int8", dtype, lengths, new, 32, 16, heads, kv, dim, pairs, interleaved, form, 1, tail=3)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", ["dense", "odd"])
@pytest.mark.parametrize("block,dim", [(128, 128), (64, 256), (128, 96), (64, 128), (128, 64), (128, 256)])
def test_blocks_of_several_pieces_a_thread(qz, fmt, dtype, form, block, dim):  # noqa: F811
    appended(qz, fmt, dtype, [300, 128, 5], [200, 1, 5], 128, block, 2, 2, dim, dim // 2, False, form, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_default_block(qz, dtype):  # noqa: F811
    cache = qz.KVCache.alloc("e4m3", 1, 1, 128, 128)
    assert cache.block == 128
    appended(qz, "e4m3", dtype, [260], [140], 128, cache.block, 4, 1, 128, 64, False, "slice", 3)


@pytest.mark.parametrize("dtype,form", [("bf16", "dense"), ("f32", "odd")])
@pytest.mark.parametrize("seqs,most", [(300, 2), (600, 3)])
def test_append_to_more_sequences_than_threads(qz, dtype, form, seqs, most):  # noqa: F811
    """300: up to 255 tokens or more, queries beside keys and values or apart; sequences without tokens among them."""
    rng = np.random.default_rng(4)
    new = [int(n) for n in rng.integers(0, most + 1, seqs)]
    lengths = [n + int(h) for n, h in zip(new, rng.integers(0, 40, seqs))]
    appended(qz, "e5m2", dtype, lengths, new, 16, 16, 2, 1, 32, 16, False, form, 4, tail=2)
    few = [1 if i % 3 == 0 else 0 for i in range(seqs)]  # fewer than 256 tokens
    appended(qz, "e5m2", dtype, [n + 20 for n in few], few, 16, 16, 2, 1, 32, 16, False, form, 5)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_tiles_of_more_sequences_than_threads(qz, fmt):  # noqa: F811
    """700 sequences of 40 or 80 rows each (some without), a kv head: the tcgen05 tiles' second look at the starts."""
    rng = np.random.default_rng(6)
    seqs, page, block, heads, kv, dim = 700, 16, 16, 40, 1, 32
    new = [int(n) for n in rng.integers(0, 3, seqs)]
    new[:3] = [1, 2, 1]
    lengths = [n + int(h) for n, h in zip(new, rng.integers(0, 30, seqs))]
    pages = [-(-n // page) for n in lengths]
    host = U.Cache(rng, fmt, sum(pages), kv, page, dim, block)
    table, at = np.full((seqs, 4), -1, np.int32), 0
    for s, n in enumerate(pages):
        table[s, :n] = np.arange(at, at + n)
        at += n
        host.fill(rng, table[s], lengths[s])
    starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    q = U.bf16(rng.standard_normal((starts[-1], heads, dim)).astype(np.float32))
    assert starts[-1] * heads > 32 * seqs
    out, lse = qz.cache_attention(gpu(q).bfloat16(), on_gpu(qz, host), gpu(table), gpu(np.array(lengths, np.int32)), gpu(starts), lse=True)
    check(out, lse, U.attention(q.astype(np.float64), host, table, lengths, starts, dim ** -0.5))
