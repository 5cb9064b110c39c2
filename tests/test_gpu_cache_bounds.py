"""The calls around the 8-bit cache with starts that are out of order: whatever is computed, nothing outside the call's rows
and the sequences' pages is written.  (Where the tiles lie: test_cache_rows.py, on the host.)"""
import numpy as np
import pytest

import cache_util as U
from test_gpu_cache import gpu, on_gpu, qz, sequences, table_of  # noqa: F401

pytestmark = pytest.mark.gpu

STARTS = [(128, (128, 0, 2)), (300, (0, 200, 100, 200)), (300, (300, 0, 150, 300)), (400, (400, 0, 0, 0)), (400, (0, 400, 0, 0, 0)),
          (400, (0, 130, 400, 0, 0)), (9, (9, 0, 3, 1)), (9, (5, 3, 1, 9))]


def framed(tokens, heads, dim, heads_outside, dtype):
    """A view [tokens, heads, dim] and the buffer around it, all 7."""
    import torch
    pad = 4 * heads * max(dim, 1) * 4
    n = tokens * heads * dim
    room = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device="cuda")
    flat = room[pad:pad + n]
    return flat.view(heads, tokens, dim).transpose(0, 1) if heads_outside else flat.view(tokens, heads, dim), room, pad


@pytest.mark.parametrize("heads_outside", [False, True])
@pytest.mark.parametrize("case", range(len(STARTS)))
@pytest.mark.parametrize("heads,kv,dim,held", [(32, 8, 64, 200), (8, 2, 128, 200), (8, 2, 64, 3000), (16, 4, 48, 1400)])
def test_starts_out_of_order(qz, case, heads_outside, heads, kv, dim, held):  # noqa: F811
    import torch
    tokens, starts = STARTS[case]
    rng = np.random.default_rng(case)
    seqs, page, block = len(starts) - 1, 32, 16
    lengths = [held + 50 * s for s in range(seqs)]
    each = -(-(max(lengths)) // page)
    host = U.Cache(rng, "e4m3", seqs * each + 3, kv, page, dim, block, junk=False)
    table = sequences(rng, seqs, each, host.pages)
    for s in range(seqs):
        host.fill(rng, table[s], lengths[s])
    cache, t = on_gpu(qz, host), gpu(table)
    n, st = gpu(np.array(lengths, np.int32)), gpu(np.array(starts, np.int32))
    owned = np.zeros(tokens, bool)
    for a, b in zip(starts, starts[1:]):
        owned[a:b] = True
    owned = gpu(owned)
    q, q_room, _ = framed(tokens, heads, dim, heads_outside, torch.bfloat16)
    q_room.copy_(torch.randn(q_room.shape, device="cuda"))
    out, room, pad = framed(tokens, heads, dim, heads_outside, torch.bfloat16)
    lse = torch.full((tokens + 8, heads), 7.0, device="cuda")
    qz.cache_attention(q, cache, t, n, st, lse=True, out=(out, lse[4:4 + tokens]))
    turned, turned_room, _ = framed(tokens, heads, dim, heads_outside, torch.bfloat16)
    spare = [b[[i for i in range(host.pages) if i not in table]].clone() for b in cache.buffers]
    cos, sin = table_of(max(lengths), dim // 2)
    k = torch.randn(tokens, kv, dim, device="cuda").bfloat16()
    qz.cache_append(cache, k, k, t, n, st, rotary=qz.RotaryTable(gpu(cos), gpu(sin)), q=q, out=turned)
    torch.cuda.synchronize()
    for view, around in ((out, room), (turned, turned_room)):
        assert (around[:pad] == 7).all() and (around[-pad:] == 7).all()
        assert (view[~owned] == 7).all()
    assert (lse[:4] == 7).all() and (lse[-4:] == 7).all() and (lse[4:-4][~owned] == 7).all()
    for b, s in zip(cache.buffers, spare):
        assert torch.equal(b[[i for i in range(host.pages) if i not in table]], s)


@pytest.mark.parametrize("lengths,new,heads", [([300, 70, 40], [1, 2, 1], 8), ([200, 140, 90], [90, 31, 60], 8), ([2600, 0, 900], [300, 0, 257], 4),
                                               ([3000, 17], [1, 1], 8)])
def test_rows_around_the_sequences_are_left_alone(qz, lengths, new, heads):  # noqa: F811
    """Rows in front of the first sequence and behind the last one; the others as if they were the whole call."""
    import torch
    rng = np.random.default_rng(8)
    page, block, kv, dim, front, back, seqs = 32, 16, 2, 64, 5, 3, len(lengths)
    each = -(-max(lengths) // page)
    host = U.Cache(rng, "int8", seqs * each, kv, page, dim, block, junk=False)
    table = sequences(rng, seqs, each, host.pages)
    for s in range(seqs):
        host.fill(rng, table[s], lengths[s])
    tokens, starts = sum(new), np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    t, n = gpu(table), gpu(np.array(lengths, np.int32))
    q, k = (torch.randn(front + tokens + back, h, dim, device="cuda").bfloat16() for h in (heads, kv))
    inner = slice(front, front + tokens)
    cos, sin = table_of(max(lengths), 32)
    rot, got = qz.RotaryTable(gpu(cos), gpu(sin)), []
    for all_rows in (False, True):
        cache, rows = on_gpu(qz, host), slice(None) if all_rows else inner
        st = gpu(starts + (front if all_rows else 0))
        turned, out = torch.full_like(q[rows], 7.0), torch.full_like(q[rows], 7.0)
        lse = torch.full(out.shape[:2], 7.0, device="cuda")
        qz.cache_append(cache, k[rows], k[rows], t, n, st, rotary=rot, q=q[rows], out=turned)
        qz.cache_attention(turned, cache, t, n, st, lse=True, out=(out, lse))
        if all_rows:
            for x in (turned, out, lse):
                assert (x[:front] == 7).all() and (x[front + tokens:] == 7).all()
            turned, out, lse = turned[inner], out[inner], lse[inner]
        got.append((turned, out, lse, *cache.buffers))
    for a, b in zip(*got):
        assert torch.equal(a, b)
