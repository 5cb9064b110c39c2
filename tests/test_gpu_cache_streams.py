"""Calls around the 8-bit cache on a stream whose earlier work they wait for: their inputs are written there, late.  (Which
stream their temporaries come from: test_cache_streams.py.)"""
import numpy as np
import pytest

from test_gpu_cache import decode_state, qz  # noqa: F401

pytestmark = pytest.mark.gpu


def late(side, pairs):
    """On `side`, after a pause: every tensor gets its value."""
    import torch
    with torch.cuda.stream(side):
        torch.cuda._sleep(60_000_000)   # some 30 ms: the calls are all made before it ends
        for t, value in pairs:
            t.copy_(value)


@pytest.mark.parametrize("call", ["rotary", "rotary_backward", "cache_append", "attention, cut", "attention, prompt"])
def test_calls_run_behind_their_streams_work(qz, call):  # noqa: F811
    import torch
    new = [200, 31] if call == "attention, prompt" else None
    host, cache, table, lengths, starts, q = decode_state(qz, [3900, 2500], new=new)
    rot = qz.RotaryTable.make(4096, qz.rotary_turns(32))
    gen = torch.Generator(device="cuda").manual_seed(7)
    k, v = (torch.randn(q.shape[0], 2, 64, device="cuda", generator=gen).bfloat16() for _ in range(2))
    positions = torch.randint(0, 4096, (q.shape[0],), device="cuda", dtype=torch.int32, generator=gen)
    st = starts if new else None

    def run(stream=None):
        if call == "cache_append":
            return (qz.cache_append(cache, k, v, table, lengths, st, rotary=rot, q=q, stream=stream), *(b.clone() for b in cache.buffers)) if stream is None else \
                (qz.cache_append(cache, k, v, table, lengths, st, rotary=rot, q=q, stream=stream),)
        if call.startswith("attention"):
            return qz.cache_attention(q, cache, table, lengths, st, lse=True, stream=stream)
        return (getattr(qz, call)(q, rot, positions, stream=stream),)

    fresh = [b.clone() for b in cache.buffers]
    want = [t.clone() for t in run()]
    for b, f in zip(cache.buffers, fresh):
        b.copy_(f)
    inputs = [q, k, v, positions, lengths, table]
    right = [t.clone() for t in inputs]
    for t in (q, k, v):
        t.normal_(generator=gen)
    positions.zero_()
    lengths.copy_(torch.tensor([300, 250], dtype=torch.int32))   # (still valid)
    table.copy_(table.flip(0))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late(side, zip(inputs, right))
    got = run(side)
    torch.cuda.synchronize()
    got = [*got, *cache.buffers] if call == "cache_append" else got
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert np.isfinite(got[0].float().cpu().numpy()).all()
