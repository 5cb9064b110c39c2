"""Rotary positions, appending to the paged 8-bit cache (both to the bit) and attention to it, on the
GPU against plain numpy."""
import numpy as np
import pytest

import cache_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qz():
    import __graft_entry__
    __graft_entry__.build_library()
    import precision_quantization_gb300 as qz
    return qz


def gpu(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def table_of(positions, pairs, seed=0):
    rng = np.random.default_rng(seed)
    angle = rng.uniform(-40, 40, (positions, pairs))
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def same_bits(a, b):
    a, b = np.ascontiguousarray(a, np.float32), np.ascontiguousarray(b, np.float32)
    return np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[~np.isnan(a)].view(np.uint32), b[~np.isnan(b)].view(np.uint32))


# ---- rotary ---------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,pairs", [(1, 1, 16, 8), (3, 5, 128, 64), (7, 9, 80, 20), (33, 2, 64, 16),
                                                    (2, 3, 7, 3), (5, 4, 256, 128), (4, 1, 96, 0), (3, 70, 48, 8), (2, 2, 34, 17)])
@pytest.mark.parametrize("form", ["dense", "slice", "heads outside", "odd"])
def test_rotary(qz, dtype, interleaved, tokens, heads, dim, pairs, form):
    import torch
    rng = np.random.default_rng(tokens * 1000 + dim)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = rng.standard_normal((tokens, heads, dim)).astype(np.float32)
    x = U.bf16(x) if dtype == "bf16" else x
    cos, sin = table_of(50, pairs)
    positions = rng.integers(0, 50, tokens).astype(np.int32)
    positions[-1] = 50 if tokens > 2 else positions[-1]   # outside the table
    if tokens > 3:
        positions[0] = -1
    t = gpu(x, dt)
    if form == "slice":
        big = torch.zeros(tokens, heads + 3, dim + 16, dtype=dt, device="cuda")
        big[:, 2:2 + heads, :dim] = t
        t = big[:, 2:2 + heads, :dim]
    elif form == "heads outside":
        t = t.transpose(0, 1).contiguous().transpose(0, 1)
    elif form == "odd":
        flat = torch.zeros(1 + t.numel(), dtype=dt, device="cuda")
        flat[1:] = t.reshape(-1)
        t = flat[1:].view(tokens, heads, dim)
    table = qz.RotaryTable(gpu(cos), gpu(sin), interleaved)
    inside = (positions >= 0) & (positions < 50)
    at = np.where(inside, positions, 0)
    for back, call in ((False, qz.rotary), (True, qz.rotary_backward)):
        want = U.rotated(x, cos[at][:, None], sin[at][:, None], interleaved, back)
        want[~inside, :, :2 * pairs] = np.nan
        want = U.bf16(want) if dtype == "bf16" else want
        assert same_bits(call(t, table, gpu(positions)).float().cpu().numpy(), want)
        want0 = U.rotated(x, cos[:tokens][:, None], sin[:tokens][:, None], interleaved, back)
        got = call(t, table)
        assert same_bits(got.float().cpu().numpy(), U.bf16(want0) if dtype == "bf16" else want0)
        mine = t.clone()
        assert call(mine, table, gpu(positions), out=mine) is mine
        assert same_bits(mine.float().cpu().numpy(), want)


def test_rotary_gradient_by_differences(qz):
    """The rotation is linear: (f(x + e) - f(x - e)) . w / 2 = f'(w) . e, fp32 sums of 2 x 48 products."""
    import torch
    rng = np.random.default_rng(5)
    x, w, e = (rng.standard_normal((6, 3, 48)).astype(np.float32) for _ in range(3))
    cos, sin = table_of(6, 16, 1)
    table = qz.RotaryTable(gpu(cos), gpu(sin))
    d = (qz.rotary(gpu(x + e), table).double() - qz.rotary(gpu(x - e), table).double()).cpu().numpy() / 2
    g = qz.rotary_backward(gpu(w), table).double().cpu().numpy()
    # three roundings an element on either side, of values up to |x| + |e| and |w|
    tol = 4 * 2.0 ** -24 * ((np.abs(x) + 2 * np.abs(e)) @ np.ones((48, 48)) * np.abs(w)).sum()
    assert abs((d * w).sum() - (g * e).sum()) <= tol
    assert torch.cuda.current_stream().query() in (True, False)


def test_rotary_table_fill(qz):
    turns = qz.rotary_turns(32, base=10000.0, scaling="parts", factor=4.0, original=512).numpy()
    table = qz.RotaryTable.make(70001, turns, amplitude=1.25)
    cos, sin = (t.cpu().numpy() for t in table.buffers)
    p = np.array([0, 1, 2, 4095, 65536, 70000])
    angle = p[:, None] * turns
    # fp32 rounding (2^-24), and 64-bit functions and angles of up to 7e4 (2^-36)
    for got, f in ((cos, np.cos), (sin, np.sin)):
        want = 1.25 * f(angle)
        assert np.abs(got[p] - want).max() <= 1.25 * (2.0 ** -24 + 2.0 ** -36)


# ---- append ---------------------------------------------------------------------------------
def sequences(rng, seqs, pages_each, pages):
    table = rng.permutation(pages)[:seqs * pages_each].reshape(seqs, pages_each).astype(np.int32)
    return table


def on_gpu(qz, c: U.Cache):
    return qz.KVCache(gpu(c.codes[0]), gpu(c.scales[0]), gpu(c.codes[1]), gpu(c.scales[1]), c.fmt)


def same_cache(got, want: U.Cache):
    for a, b in zip(got.buffers, (want.codes[0], want.scales[0], want.codes[1], want.scales[1])):
        a = a.cpu().numpy()
        if a.dtype == np.float32:
            assert same_bits(a, b)
        else:
            assert np.array_equal(a, b), np.argwhere(a != b)[:4]


APPEND = [  # lengths after, new tokens, page, block, heads, kv, dim, pairs
    ([1], [1], 16, 16, 4, 2, 64, 32),
    ([17, 16, 15, 33], [1, 1, 1, 1], 16, 16, 8, 2, 128, 64),
    ([40, 64, 65], [1, 1, 1], 64, 32, 3, 3, 80, 20),
    ([50, 7, 0, 129, 64], [50, 3, 0, 128, 1], 64, 64, 4, 1, 96, 48),
    ([300, 5], [129, 5], 128, 128, 2, 1, 256, 128),
    ([37, 90], [30, 2], 32, 16, 4, 4, 48, 9),
    ([4, 40], [9, 45], 48, 16, 2, 2, 16, 8),      # more new tokens than the length: the first lie below 0
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(APPEND)))
@pytest.mark.parametrize("interleaved,form", [(False, "dense"), (True, "slice"), (False, "odd")])
def test_append(qz, fmt, dtype, case, interleaved, form):
    import torch
    lengths, new, page, block, heads, kv, dim, pairs = APPEND[case]
    rng = np.random.default_rng(case)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    seqs, tokens = len(lengths), sum(new)
    each = -(-max(lengths + [1]) // page)
    host = U.Cache(rng, fmt, seqs * each + 2, kv, page, dim, block)
    table = sequences(rng, seqs, each, host.pages)
    for s in range(seqs):
        host.fill(rng, table[s], max(lengths[s] - new[s], 0))
    if case == 3:
        table[3, 1] = -1          # a token with no page
        table[0, 0] = host.pages  # and outside the cache
    rnd = lambda *s: (lambda v: U.bf16(v) if dtype == "bf16" else v)((1.5 * rng.standard_normal(s)).astype(np.float32))  # noqa: E731
    k, v, q = rnd(tokens, kv, dim), rnd(tokens, kv, dim), rnd(tokens, heads, dim)
    cos, sin = table_of(max(lengths) - (1 if case == 3 else 0), pairs)   # case 3: one position outside the table
    starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    tk, tv, tq = (gpu(a, dt) for a in (k, v, q))
    if form == "slice":  # views of one fused projection
        fused = torch.cat((tq, tk, tv), 1)
        tq, tk, tv = fused[:, :heads], fused[:, heads:heads + kv], fused[:, heads + kv:]
    elif form == "odd":
        shift = lambda t: torch.cat((t.new_zeros(1), t.reshape(-1)))[1:].view(t.shape)  # noqa: E731
        tq, tk, tv = shift(tq), shift(tk), shift(tv)
    cache = on_gpu(qz, host)
    rot = qz.RotaryTable(gpu(cos), gpu(sin), interleaved)
    one = all(n == 1 for n in new)
    got = qz.cache_append(cache, tk, tv, gpu(table), gpu(np.array(lengths, np.int32)), None if one else gpu(starts), rotary=rot, q=tq)
    host.append(k, v, table, lengths, starts, cos, sin, interleaved)
    same_cache(cache, host)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lengths, new)])
    inside = (pos >= 0) & (pos < len(cos))
    at = np.where(inside, pos, 0)
    want = U.rotated(q, cos[at][:, None], sin[at][:, None], interleaved)
    want[~inside, :, :2 * pairs] = np.nan
    assert same_bits(got.float().cpu().numpy(), U.bf16(want) if dtype == "bf16" else want)
    # in place, and without a rotation
    mine = tq.clone()
    qz.cache_append(cache, tk, tv, gpu(table), gpu(np.array(lengths, np.int32)), None if one else gpu(starts), rotary=rot, q=mine, out=mine)
    assert torch.equal(mine.view(torch.int16 if dtype == "bf16" else torch.int32), got.view(torch.int16 if dtype == "bf16" else torch.int32))
    assert qz.cache_append(cache, tk, tv, gpu(table), gpu(np.array(lengths, np.int32)), None if one else gpu(starts)) is None
    host.append(k, v, table, lengths, starts, cos, sin, interleaved)
    host.append(k, v, table, lengths, starts, None, None, interleaved)
    same_cache(cache, host)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
def test_append_token_by_token(qz, fmt):
    """The scale of a block grows with its tokens; zeros first, then larger and larger values, one NaN."""
    rng = np.random.default_rng(3)
    host = U.Cache(rng, fmt, 4, 2, 32, 32, 16)
    cache = on_gpu(qz, host)
    table = np.array([[2, 0]], np.int32)
    for n in range(1, 50):
        size = 0.0 if n < 4 else 2.0 ** (n % 16 - 6) if n < 40 else 1e-30 if n < 44 else 1e30
        k, v = (U.bf16(size * rng.standard_normal((1, 2, 32)).astype(np.float32)) for _ in range(2))
        if n == 23:
            k[0, 1, 5], v[0, 0, 7] = np.nan, np.inf
        qz.cache_append(cache, *(gpu(a).bfloat16() for a in (k, v)), gpu(table), gpu(np.array([n], np.int32)))
        host.append(k, v, table, [n], [0, 1], None, None, False)
        same_cache(cache, host)


def test_append_leaves_other_rows(qz):
    """Rows behind the last sequence and sequences without new tokens: nothing is written."""
    import torch
    rng = np.random.default_rng(1)
    host = U.Cache(rng, "int8", 4, 1, 16, 16, 16)
    cache = on_gpu(qz, host)
    cos, sin = table_of(64, 8)
    k, v, q = (rng.standard_normal((9, 1, 16)).astype(np.float32) for _ in range(3))
    table, starts = np.array([[1], [3], [0]], np.int32), np.array([0, 2, 2, 5], np.int32)
    out = torch.full((9, 1, 16), 7.0, device="cuda")
    qz.cache_append(cache, gpu(k), gpu(v), gpu(table), gpu(np.array([2, 9, 3], np.int32)), gpu(starts),
                    rotary=qz.RotaryTable(gpu(cos), gpu(sin)), q=gpu(q), out=out)
    host.append(k, v, table, [2, 9, 3], starts, cos, sin, False)
    same_cache(cache, host)
    assert (out[5:] == 7).all() and not (out[:5] == 7).any()


# ---- attention ------------------------------------------------------------------------------
ATTEND = [  # lengths, new tokens, page, block, heads, kv, dim, window
    ([1], [1], 16, 16, 1, 1, 16, 0),
    ([5, 16, 17, 0, 200], [1, 1, 1, 1, 1], 16, 16, 8, 2, 64, 0),
    ([700, 64, 65, 511], [1, 1, 1, 1], 64, 32, 24, 3, 128, 0),
    ([300, 129], [1, 1], 128, 128, 20, 4, 96, 50),
    ([257, 100], [1, 1], 32, 32, 71, 1, 80, 0),
    ([150, 90], [1, 1], 16, 16, 4, 2, 256, 0),
    ([130, 40], [1, 1], 48, 16, 6, 2, 192, 1),
    ([60, 33, 300, 5], [3, 0, 7, 5], 32, 16, 5, 1, 64, 0),
    ([190, 256, 30], [40, 131, 30], 64, 64, 8, 2, 128, 0),
    ([333, 20], [200, 20], 32, 32, 4, 2, 64, 17),
    ([100, 6], [3, 9], 16, 16, 4, 4, 48, 0),     # more new tokens than the length: the first see nothing
    ([400], [260], 128, 64, 2, 2, 112, 300),
    ([290, 300], [70, 45], 128, 128, 16, 1, 128, 0),
    ([140], [77], 16, 16, 6, 2, 240, 60),
    # too long for one CTA: cut and joined
    ([3000, 17, 1111, 0], [1, 1, 1, 1], 64, 32, 16, 2, 128, 0),
    ([2500, 0, 1800], [3, 0, 2], 32, 16, 12, 2, 64, 700),
    ([5000], [1], 128, 64, 4, 1, 256, 0),
    ([1300, 2100], [9, 4], 16, 16, 8, 2, 128, 0),
    ([1100, 40], [150, 40], 32, 32, 4, 2, 96, 0),
    ([2600, 0, 900], [300, 0, 257], 64, 64, 8, 1, 128, 0),
    ([2000], [130], 32, 16, 4, 4, 64, 200),
    ([700, 1300], [100, 90], 48, 16, 6, 2, 80, 0),
    ([600], [1000], 64, 64, 2, 2, 16, 0),
]


def attend(qz, fmt, case, spread=1.0, seed=0, mask=False):
    lengths, new, page, block, heads, kv, dim, window = case
    rng = np.random.default_rng(seed + dim + len(lengths))
    seqs, tokens = len(lengths), sum(new)
    each = -(-max(lengths + [1]) // page)
    host = U.Cache(rng, fmt, seqs * each + 1, kv, page, dim, block)
    table = sequences(rng, seqs, each, host.pages)
    for s in range(seqs):
        host.fill(rng, table[s], lengths[s], spread)
        table[s, -(-lengths[s] // page):] = -1 if s % 2 else 1 << 30
    if mask:
        table[0, 0] = -5
    q = U.bf16((2 * rng.standard_normal((tokens, heads, dim))).astype(np.float32))
    starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    return host, table, q, starts


def check(out, lse, want, what=""):
    ref, ref_lse = want[:2]
    tol, tol_lse = U.attention_tolerance(*want)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(out).all()
    worst = float(np.max(np.abs(out - ref) / np.maximum(tol, 1e-300)))
    assert worst <= 1, (what, worst)
    none = np.isinf(ref_lse)
    assert np.array_equal(lse[none], ref_lse[none]) and (out[none] == 0).all()
    worst = float(np.max(np.abs(lse[~none] - ref_lse[~none]) / tol_lse[~none], initial=0))
    assert worst <= 1, (what, worst)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention(qz, fmt, case):
    lengths, new, page, block, heads, kv, dim, window = ATTEND[case]
    host, table, q, starts = attend(qz, fmt, ATTEND[case])
    cache, scale = on_gpu(qz, host), dim ** -0.5
    one = all(n == 1 for n in new)
    args = (gpu(q).bfloat16(), cache, gpu(table), gpu(np.array(lengths, np.int32)), None if one else gpu(starts))
    out, lse = qz.cache_attention(*args, window=window or None, lse=True)
    check(out, lse, U.attention(q.astype(np.float64), host, table, lengths, starts, scale, window))
    again = qz.cache_attention(*args, window=window or None)
    assert (again.view(__import__("torch").int16) == out.view(__import__("torch").int16)).all()
    if one:  # the same with starts
        out2, lse2 = qz.cache_attention(*args[:4], gpu(starts), window=window or None, lse=True)
        check(out2, lse2, U.attention(q.astype(np.float64), host, table, lengths, starts, scale, window))


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("case", [2, 8, 12])
def test_attention_scales_far_apart(qz, fmt, case):
    """Blocks whose scales differ by factors of thousands, a page that is missing, sharp scores."""
    lengths, new, page, block, heads, kv, dim, window = ATTEND[case]
    host, table, q, starts = attend(qz, fmt, ATTEND[case], spread=3.0, seed=9, mask=True)
    for s in range(len(lengths)):   # and a block of zeros
        if lengths[s] > 2 * block and table[s, (lengths[s] - 1) // page] >= 0:
            for c, z in zip(host.codes, host.scales):
                c[table[s, 1 * block // page], :, block % page:block % page + block] = 0
                z[table[s, 1 * block // page], :, block % page // block] = 0
    scale = 0.02
    out, lse = qz.cache_attention(gpu(q).bfloat16(), on_gpu(qz, host), gpu(table), gpu(np.array(lengths, np.int32)), gpu(starts),
                                  scale=scale, window=window or None, lse=True)
    check(out, lse, U.attention(q.astype(np.float64), host, table, lengths, starts, scale, window))


@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -60, 2.0 ** 100])
def test_attention_queries_of_any_size(qz, size):
    lengths, new, page, block, heads, kv, dim, window = ATTEND[8]
    host, table, q, starts = attend(qz, "e4m3", ATTEND[8])
    q[1::3] *= np.float32(size)
    scale = float(dim ** -0.5 / max(size, 1.0))
    for some in (slice(None), slice(0, 40)):
        n = [40] if some.stop else new
        st = np.concatenate(([0], np.cumsum(n))).astype(np.int32)
        out, lse = qz.cache_attention(gpu(q[some]).bfloat16(), on_gpu(qz, host), gpu(table[:len(n)]), gpu(np.array(lengths[:len(n)], np.int32)),
                                      gpu(st), scale=scale, lse=True)
        check(out, lse, U.attention(q[some].astype(np.float64), host, table, lengths[:len(n)], st, scale))


@pytest.mark.parametrize("case", [2, 8])
def test_attention_non_finite_query(qz, case):
    lengths, new, page, block, heads, kv, dim, window = ATTEND[case]
    host, table, q, starts = attend(qz, "int8", ATTEND[case])
    args = (on_gpu(qz, host), gpu(table), gpu(np.array(lengths, np.int32)), gpu(starts))
    want = qz.cache_attention(gpu(q).bfloat16(), *args).float().cpu().numpy()
    q[1, 2, 3], q[2, 1, 0] = np.nan, np.inf
    got = qz.cache_attention(gpu(q).bfloat16(), *args).float().cpu().numpy()
    bad = np.zeros(want.shape[:2], bool)
    bad[1, 2] = bad[2, 1] = True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], want[~bad])


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2"])
@pytest.mark.parametrize("new", [1, 90])
def test_attention_sees_no_later_spoiled_block(qz, fmt, new):
    """A block with a NaN scale (its new values were not finite) spoils the rows that see it, no others."""
    lengths, page, block, heads, kv, dim = [200], 64, 16, 4, 2, 64
    host, table, q, starts = attend(qz, fmt, (lengths, [new], page, block, heads, kv, dim, 0))
    at = 160 if new > 1 else 16
    for c, z in zip(host.codes, host.scales):
        z[table[0, at // page], 1, at % page // block] = np.nan
        c[table[0, at // page], 1, at % page:at % page + block] = 0
    got = qz.cache_attention(gpu(q).bfloat16(), on_gpu(qz, host), gpu(table), gpu(np.array(lengths, np.int32)), gpu(starts)).float().cpu().numpy()
    pos = np.arange(200 - new, 200)
    bad = np.zeros((new, heads), bool)
    bad[pos >= at, heads // kv:] = True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


@pytest.mark.parametrize("new", [[3, 2, 40], [1, 2, 1]])
def test_attention_strides_and_padding(qz, new):
    """Queries and outputs as slices, heads outside tokens; rows behind the last sequence stay."""
    import torch
    case = ([60, 33, 100], new, 32, 16, 6, 2, 64, 0)
    lengths, new, page, block, heads, kv, dim, window = case
    host, table, q, starts = attend(qz, "e4m3", case)
    tokens = sum(new)
    cache, t, n, st = on_gpu(qz, host), gpu(table), gpu(np.array(lengths, np.int32)), gpu(starts)
    want, wl = qz.cache_attention(gpu(q).bfloat16(), cache, t, n, st, lse=True)
    for pad, make in ((16, lambda *s: torch.full((s[0], s[1] + 2, s[2] + 16), 7.0, dtype=torch.bfloat16, device="cuda")[:, 1:1 + s[1], :s[2]]),
                      (3, lambda *s: torch.full((s[1], s[0], s[2] + 1), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[..., :s[2]])):
        qq, out = make(tokens + 5, heads, dim), make(tokens + 5, heads, dim)
        qq[:tokens] = gpu(q).bfloat16()
        logs = torch.full((tokens + 5, heads + 1), 7.0, device="cuda")[:, :heads]
        qz.cache_attention(qq, cache, t, n, st, lse=True, out=(out, logs))
        assert torch.equal(out[:tokens], want) and torch.equal(logs[:tokens], wl)
        assert (out[tokens:] == 7).all() and (logs[tokens:] == 7).all()


def test_append_then_attend(qz):
    """A prompt, then tokens one by one: each call's outputs against the reference on the cache so far."""
    rng = np.random.default_rng(2)
    fmt, page, block, heads, kv, dim, pairs = "e4m3", 32, 16, 8, 2, 64, 32
    host = U.Cache(rng, fmt, 12, kv, page, dim, block)
    cache = on_gpu(qz, host)
    cos, sin = table_of(200, pairs, 4)
    rot = qz.RotaryTable(gpu(cos), gpu(sin))
    table, lengths = np.array([[3, 7, 1, 9], [2, 0, 5, 11]], np.int32), np.array([0, 0])
    for new in ([70, 45], [1, 1], [1, 1], [0, 3], [1, 1], [20, 1], [1, 1]):
        lengths = lengths + new
        tokens, starts = sum(new), np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        k, v, q = (U.bf16(rng.standard_normal((tokens, n, dim)).astype(np.float32)) for n in (kv, kv, heads))
        t, n, st = gpu(table), gpu(lengths.astype(np.int32)), None if new == [1, 1] else gpu(starts)
        qr = qz.cache_append(cache, gpu(k).bfloat16(), gpu(v).bfloat16(), t, n, st, rotary=rot, q=gpu(q).bfloat16())
        out, lse = qz.cache_attention(qr, cache, t, n, st, lse=True)
        host.append(k, v, table, lengths, starts, cos, sin, False)
        same_cache(cache, host)
        check(out, lse, U.attention(qr.double().cpu().numpy(), host, table, list(lengths), starts, dim ** -0.5))


# ---- streams, graphs, many calls at once --------------------------------------------------------
def decode_state(qz, lengths, fmt="int8", new=None, page=32, block=16, heads=8, kv=2, dim=64, capacity=4096):
    """A cache with room for `capacity` tokens a sequence, and the tensors of one step."""
    rng = np.random.default_rng(len(lengths))
    new = new or [1] * len(lengths)
    each = capacity // page
    host = U.Cache(rng, fmt, len(lengths) * each, kv, page, dim, block, junk=False)
    table = sequences(rng, len(lengths), each, host.pages)
    for s, n in enumerate(lengths):
        host.fill(rng, table[s], n)
    q = U.bf16(rng.standard_normal((sum(new), heads, dim)).astype(np.float32))
    starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    return host, on_gpu(qz, host), gpu(table), gpu(np.array(lengths, np.int32)), gpu(starts), gpu(q).bfloat16()


@pytest.mark.parametrize("new", [None, [70, 40, 90]])
def test_captured_once_replayed_as_the_sequences_grow(qz, new):
    """Append and attention in one graph: lengths and tables are read on the GPU at each replay."""
    import torch
    lengths = [300, 1700, 33] if new is None else [300, 1700, 133]
    host, cache, table, n, starts, q = decode_state(qz, lengths, new=new)
    st = None if new is None else starts
    tokens = q.shape[0]
    table_r = qz.RotaryTable.make(4096, qz.rotary_turns(32))
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(tokens, 2, 64, device="cuda", generator=gen).bfloat16() for _ in range(2))

    def step():
        qr = qz.cache_append(cache, k, v, table, n, st, rotary=table_r, q=q)
        return qz.cache_attention(qr, cache, table, n, st, lse=True)

    fresh = [b.clone() for b in cache.buffers]
    step()
    for b, f in zip(cache.buffers, fresh):
        b.copy_(f)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = step()
    got = []
    for _ in range(3):
        graph.replay()
        got.append((out.clone(), lse.clone()))
        n += 1 if new is None else 100
    replayed = [b.clone() for b in cache.buffers]
    for b, f in zip(cache.buffers, fresh):
        b.copy_(f)
    n -= 3 if new is None else 300
    for o, s in got:
        want, wl = step()
        assert torch.equal(o, want) and torch.equal(s, wl)
        n += 1 if new is None else 100
    assert all(torch.equal(a, b) for a, b in zip(replayed, cache.buffers))


def test_two_streams_at_once(qz):
    """Calls that overlap have a workspace each: long sequences (partial results) on one stream, prompts on the
    other, and both again after each other."""
    import torch
    a = decode_state(qz, [4000, 3000], capacity=4096)
    b = decode_state(qz, [3500], new=[200], fmt="e4m3")
    call = lambda s, st, **k: qz.cache_attention(s[5], s[1], s[2], s[3], st, lse=True, **k)  # noqa: E731
    want = call(a, None), call(b, b[4])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        got = call(a, None, stream=side), call(b, b[4])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_rotary_and_append_on_a_busy_side_stream(qz):
    import torch
    host, cache, table, n, starts, q = decode_state(qz, [100, 40])
    rot = qz.RotaryTable.make(200, qz.rotary_turns(32))
    k = torch.randn(2, 2, 64, device="cuda").bfloat16()
    want_q = qz.cache_append(cache, k, k, table, n, rotary=rot, q=q)
    want_r = qz.rotary(q, rot)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000)
    got_q = qz.cache_append(cache, k, k, table, n, rotary=rot, q=q, stream=side)
    got_r = qz.rotary(q, rot, stream=side)
    torch.full((q.numel() * 2,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(got_q, want_q) and torch.equal(got_r, want_r)


def test_positions_past_the_table_and_bad_starts(qz):
    """A length beyond what the table's pages hold, starts that decrease or pass the rows: nothing outside the
    tensors is touched, and what is inside is as if they ended there."""
    import torch
    for new in ([1, 1], [40, 40]):
        host, cache, table, n, starts, q = decode_state(qz, [64, 64], new=new, capacity=64)
        k = torch.randn(q.shape[0], 2, 64, device="cuda").bfloat16()
        before = [b.clone() for b in cache.buffers]
        n[1] = 64 + new[1] + 5                       # sequence 1: every new token past its pages
        qz.cache_append(cache, k, k, table, n, starts)
        assert all(torch.equal(a[table[1].long()], b[table[1].long()]) for a, b in zip(cache.buffers, before))
        out = qz.cache_attention(q, cache, table, n, starts)
        assert torch.isfinite(out.float()).all()
        for bad in ([0, 5, 3], [0, -7, 1 << 30], [1 << 30, 0, 2], [-5, -4, -3]):
            st = torch.tensor(bad, dtype=torch.int32, device="cuda")
            qz.cache_append(cache, k, k, table, n, st)
            qz.cache_attention(q, cache, table, n, st, lse=True)
        torch.cuda.synchronize()


@pytest.mark.parametrize("seqs", [700])
def test_many_sequences(qz, seqs):
    """More sequences than a CTA has threads, most of them short, one long."""
    rng = np.random.default_rng(0)
    lengths = [int(x) for x in rng.integers(0, 40, seqs)]
    lengths[555] = 1500
    page, block, heads, kv, dim = 16, 16, 2, 1, 32
    host = U.Cache(rng, "e5m2", seqs * 4 + 200, kv, page, dim, block, junk=False)
    table = np.full((seqs, 200), -1, np.int32)
    at = 0
    for s, n in enumerate(lengths):
        table[s, :-(-n // page)] = np.arange(at, at + -(-n // page))
        at += -(-n // page)
        host.fill(rng, table[s], n)
    q = U.bf16(rng.standard_normal((seqs, heads, dim)).astype(np.float32))
    starts = np.arange(seqs + 1)
    want = U.attention(q.astype(np.float64), host, table, lengths, starts, dim ** -0.5)
    for width in (200, 94):   # cut into shares; whole items (the table's first columns hold every page)
        out, lse = qz.cache_attention(gpu(q).bfloat16(), on_gpu(qz, host), gpu(table)[:, :width], gpu(np.array(lengths, np.int32)), lse=True)
        check(out, lse, want, width)


@pytest.mark.parametrize("new", [[1, 1], [40, 70]])
def test_shared_pages(qz, new):
    """Sequences with the same first pages see what each would see of a copy of its own."""
    host, table, q, starts = attend(qz, "int8", ([1200, 900], new, 64, 32, 8, 2, 128, 0))
    table[1, :12] = table[0, :12]
    cache, n = on_gpu(qz, host), np.array([1200, 900], np.int32)
    out, lse = qz.cache_attention(gpu(q).bfloat16(), cache, gpu(table), gpu(n), gpu(starts), lse=True)
    check(out, lse, U.attention(q.astype(np.float64), host, table, [1200, 900], starts, 128 ** -0.5, 0))


@pytest.mark.parametrize("fmt,new", [("e4m3", [1, 1]), ("int8", [60, 90])])
def test_offsets_past_32_bits(qz, fmt, new):
    """Codes, queries, keys and outputs that lie 2^32 elements and more from their tensors' start: the same results
    as near it."""
    import torch
    far, near, kv, heads, page, dim, pairs = 70000, 64, 8, 16, 64, 128, 64   # 70000 pages: 4.6e9 codes an array
    tokens, lengths = sum(new), gpu(np.array([900, 700], np.int32))
    starts, ld = gpu(np.concatenate(([0], np.cumsum(new))).astype(np.int32)), (1 << 32) // (tokens - 1) // 64 * 64 + 64
    torch.manual_seed(5)
    room = torch.empty(((tokens - 1) * ld + heads * dim,), dtype=torch.bfloat16, device="cuda")
    wide = room.as_strided((tokens, heads, dim), (ld, dim, 1))
    table = torch.arange(30, dtype=torch.int32, device="cuda").reshape(2, 15)
    cos, sin = table_of(1000, pairs, 4)
    rot, got = qz.RotaryTable(gpu(cos), gpu(sin)), []
    q, k, v = (torch.randn((tokens, n, dim), device="cuda").bfloat16() for n in (heads, kv, kv))
    held = torch.randint(0, 120, (2, 30, kv, page, dim), dtype=torch.uint8, device="cuda")
    for pages in (near, far):
        cache, t = qz.KVCache.alloc(fmt, pages, kv, page, dim), table + (pages - 30)
        cache.k_codes[-30:], cache.v_codes[-30:] = held[0], held[1]
        cache.k_scales[-30:], cache.v_scales[-30:] = 0.01, 0.02
        if pages == near:
            turned = qz.cache_append(cache, k, v, t, lengths, starts, rotary=rot, q=q)
            out, lse = qz.cache_attention(turned, cache, t, lengths, starts, lse=True)
        else:
            wide.copy_(q)
            assert qz.cache_append(cache, k, v, t, lengths, starts, rotary=rot, q=wide, out=wide) is wide
            turned = wide.clone(memory_format=torch.contiguous_format)
            out, lse = qz.cache_attention(wide, cache, t, lengths, starts, lse=True)
            assert torch.equal(qz.rotary(wide, rot), qz.rotary(turned, rot))
            wide.copy_(q)
            kk = wide[:, :kv]
            kk.copy_(k)
            before = cache.k_codes[-30:].clone()
            qz.cache_append(cache, kk, v, t, lengths, starts, rotary=rot)
            assert torch.equal(cache.k_codes[-30:], before)
            wide.fill_(7)
            qz.cache_attention(turned, cache, t, lengths, starts, out=wide)
            assert torch.equal(wide.clone(memory_format=torch.contiguous_format), out)
        got.append((turned, out, lse, *(b[-30:].clone() for b in cache.buffers)))
        del cache
    for a, b in zip(*got):
        assert torch.equal(a, b)
