"""Measured cases of the operators around a key-value cache held in 8 bits: the rotation of
queries and keys by their positions (``rotary``, ``rotary_backward``), appending keys and values
to a paged INT8 / FP8 cache with one scale for each block of tokens and head
(``cache_append``), and the attention that reads it (``cache_attention``).

``run`` computes each in its plain form (elementary torch operations in 32 bits, rounded once
at the end), or, where ``own`` is true, by the library's calls.  ``exact`` is the definition
in 64 bits.
"""
import math

import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0, "e5m2": 57344.0}
VIEW = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the queries of one decoded token: launch latency is all there is
        dict(name="rotary 1 token", op="rotary", dtype="bf16", tokens=1, heads=32, dim=128, pairs=64, interleaved=False, positions=4096),
        # the queries of a prompt or a training batch, adjacent pairs
        dict(name="rotary 8192 tokens", op="rotary", dtype="bf16", tokens=8192, heads=32, dim=128, pairs=64, interleaved=True, positions=8192),
        # the gradient of an odd batch, a quarter of each head rotated, fp32
        dict(name="rotary backward 4093 tokens", op="rotary_backward", dtype="f32", tokens=4093, heads=40, dim=80, pairs=10, interleaved=False, positions=16384),
        # one decoded token of one sequence
        dict(name="append 1 token", op="append", fmt="e4m3", dtype="bf16", block=16, page=16, heads=32, kv_heads=8, dim=128, pairs=64, interleaved=False, seqs=1, length=777, queries=1, ragged=False),
        # one decoded token of each sequence of a large batch
        dict(name="append 128 x 1 token", op="append", fmt="int8", dtype="bf16", block=32, page=64, heads=32, kv_heads=8, dim=128, pairs=64, interleaved=False, seqs=128, length=2049, queries=1, ragged=True),
        # prompts of different lengths, continued in the middle of a block
        dict(name="append prompts", op="append", fmt="e4m3", dtype="bf16", block=64, page=64, heads=32, kv_heads=8, dim=128, pairs=64, interleaved=False, seqs=4, length=4109, queries=4096, ragged=True),
        # one token of one short sequence: latency again
        dict(name="attention 1 token", op="attention", fmt="e4m3", block=16, page=16, heads=32, kv_heads=8, dim=128, seqs=1, length=517, queries=1, ragged=False, window=0, lse=False),
        # one token of each sequence of a batch, ragged
        dict(name="attention 64 x 1 token", op="attention", fmt="int8", block=64, page=64, heads=32, kv_heads=8, dim=128, seqs=64, length=8192, queries=1, ragged=True, window=0, lse=False),
        # one token at the end of a long context
        dict(name="attention long context", op="attention", fmt="e4m3", block=32, page=128, heads=64, kv_heads=8, dim=128, seqs=1, length=131072, queries=1, ragged=False, window=0, lse=True),
        # three tokens a sequence (a drafted continuation) behind a sliding window, an odd group of heads
        dict(name="attention window 24 x 3", op="attention", fmt="e5m2", block=16, page=32, heads=40, kv_heads=8, dim=64, seqs=24, length=20011, queries=3, ragged=True, window=4096, lse=False),
        # the second half of a long prompt
        dict(name="attention prompt", op="attention", fmt="e4m3", block=64, page=64, heads=32, kv_heads=8, dim=128, seqs=1, length=8192, queries=4096, ragged=False, window=0, lse=True),
        # prompts of different, odd lengths
        dict(name="attention ragged prompts", op="attention", fmt="int8", block=32, page=32, heads=16, kv_heads=4, dim=64, seqs=5, length=3001, queries=1111, ragged=True, window=0, lse=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_backward", "append", "append", "attention", "attention", "attention"])
    dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
    pairs = rng.choice([dim // 2, dim // 2, dim // 4, dim // 8])
    interleaved = rng.choice([False, True])
    if op.startswith("rotary"):
        dtype, heads = rng.choice(["bf16", "bf16", "f32"]), _spread(rng, 1, 64)
        tokens = _spread(rng, 1, max(1, min(16384, 8192 * 32 * 128 // (heads * dim))))
        return dict(op=op, dtype=dtype, tokens=tokens, heads=heads, dim=dim, pairs=pairs, interleaved=interleaved, positions=max(tokens, 8192))
    fmt, page = rng.choice(["int8", "e4m3", "e5m2"]), rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= page])
    kv_heads, group = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 3, 4, 4, 5, 8, 8, 16])
    case = dict(op=op, fmt=fmt, block=block, page=page, heads=kv_heads * group, kv_heads=kv_heads, dim=dim)
    ragged = rng.choice([False, True, True])
    if op == "append":
        queries = rng.choice([1, _spread(rng, 2, 4096)])
        seqs = _spread(rng, 1, max(1, min(256, 8192 // queries)))
        length = queries + _spread(rng, 1, 2048)
        return dict(case, dtype=rng.choice(["bf16", "bf16", "f32"]), pairs=pairs, interleaved=interleaved, seqs=seqs, length=length, queries=queries, ragged=ragged)
    if rng.random() < 0.6:  # decoding: a few tokens a sequence, bound by the cache's bytes
        queries, length = rng.choice([1, 1, 1, rng.randint(2, 8)]), _spread(rng, 8, 131072)
        seqs = _spread(rng, 1, max(1, min(128, 500_000_000 // (length * kv_heads * dim * 2))))
    else:  # prompts
        length = _spread(rng, 64, 16384)
        queries = min(length, _spread(rng, 9, 4096))
        seqs = _spread(rng, 1, max(1, min(8, 600_000_000 // (length * queries * case["heads"] * max(1, dim // 128)))))
        queries = max(1, min(queries, 600_000_000 // (length * seqs * case["heads"] * max(1, dim // 128))))
    window = rng.choice([0, 0, _spread(rng, 1, max(2, length))])
    return dict(case, seqs=seqs, length=length, queries=queries, ragged=ragged, window=window, lse=rng.choice([False, True]))


# ---- inputs ---------------------------------------------------------------------------------
def _lengths(case):
    """Tokens of each sequence after the call, and how many of them are new."""
    length, new = [], []
    for b in range(case["seqs"]):
        n, q = case["length"], case["queries"]
        if case["ragged"]:
            n, q = n - n // 2 * (37 * b % 16) // 16, q - q * (11 * b % 8) // 12
        length.append(max(1, n))
        new.append(max(1, min(q, length[-1])))
    return length, new


def _capacity(case):
    """Pages of each sequence; a cache that grows has room for another such step."""
    more = case["queries"] + 2 * case["block"] if case["op"] == "append" else 0
    return -(-(case["length"] + more) // case["page"])


def _normal(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _round_codes(v, fmt):
    """The nearest codes of fp32 values, as bytes."""
    v = v.clamp(-QMAX[fmt], QMAX[fmt])
    return (v.round().to(torch.int8) if fmt == "int8" else v.to(VIEW[fmt])).view(torch.uint8)


def _cache(case, pages, gen):
    """Codes and scales of normal keys or values with a mean of their own in each channel."""
    heads, page, dim, block, fmt = case["kv_heads"], case["page"], case["dim"], case["block"], case["fmt"]
    codes = torch.empty(pages, heads, page, dim, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, heads, page // block, device="cuda")
    mean = 0.5 * _normal(gen, heads, 1, dim)
    step = max(1, (1 << 26) // (heads * page * dim))
    for p in range(0, pages, step):
        x = _normal(gen, min(step, pages - p), heads, page, dim) + mean
        x = x.reshape(-1, heads, page // block, block, dim)
        s = x.abs().amax((-1, -2)) / QMAX[fmt]
        scales[p:p + step] = s
        codes[p:p + step] = _round_codes(x / s[..., None, None], fmt).reshape(-1, heads, page, dim)
    return codes, scales


def _rotation(positions, pairs):
    """cos and sin of each position and pair, [positions, pairs]."""
    turn = 10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * turn
    return angle.cos().float(), angle.sin().float()


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s, op, dim = dict(case), case["op"], case["dim"]
    if op.startswith("rotary"):
        s["x"] = _normal(gen, case["tokens"], case["heads"], dim).to(DTYPE[case["dtype"]])
        s["positions"] = torch.randint(0, case["positions"], (case["tokens"],), device="cuda", dtype=torch.int32, generator=gen)
        s["cos"], s["sin"] = _rotation(case["positions"], case["pairs"])
        return s
    length, new = _lengths(case)
    capacity, tokens = _capacity(case), sum(new)
    s["lengths"] = torch.tensor(length, dtype=torch.int32, device="cuda")
    starts = [sum(new[:b]) for b in range(case["seqs"] + 1)]
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda") if case["queries"] > 1 else None
    pages = capacity * case["seqs"]
    s["table"] = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32).reshape(case["seqs"], capacity)
    s["k"], s["v"] = _cache(case, pages, gen), _cache(case, pages, gen)
    s["q"] = _normal(gen, tokens, case["heads"], dim).to(DTYPE[case.get("dtype", "bf16")])
    if op == "append":
        dt = DTYPE[case["dtype"]]
        s["new_k"], s["new_v"] = ((1.3 * _normal(gen, tokens, case["kv_heads"], dim)).to(dt) for _ in range(2))
        s["cos"], s["sin"] = _rotation(case["length"], case["pairs"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the handles that a program keeps with its cache and its table
        import precision_quantization_gb300 as qz
        if "cos" in s:
            s["rotary"] = qz.RotaryTable(s["cos"], s["sin"], interleaved=case["interleaved"])
        if "k" in s:
            s["cache"] = qz.KVCache(*s["k"], *s["v"], fmt=case["fmt"])
    return s


# ---- one pass ---------------------------------------------------------------------------------
def _run_own(s):
    import precision_quantization_gb300 as qz
    op = s["op"]
    if op == "rotary":
        return qz.rotary(s["x"], s["rotary"], s["positions"])
    if op == "rotary_backward":
        return qz.rotary_backward(s["x"], s["rotary"], s["positions"])
    if op == "append":
        q = qz.cache_append(s["cache"], s["new_k"], s["new_v"], s["table"], s["lengths"], starts=s["starts"], rotary=s["rotary"], q=s["q"])
        return _contents(s, q)
    return qz.cache_attention(s["q"], s["cache"], s["table"], s["lengths"], starts=s["starts"], window=s["window"] or None, lse=s["lse"])


def _contents(s, q):
    (kc, ks), (vc, vs), view = s["k"], s["v"], VIEW[s["fmt"]]
    return q, kc.view(view), ks, vc.view(view), vs


def _rotate(x, cos, sin, pairs, interleaved):
    """x: [..., dim], fp32; cos, sin: [..., pairs]."""
    y = x.clone()
    a, b = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if interleaved else (slice(0, pairs), slice(pairs, 2 * pairs))
    x1, x2 = x[..., a], x[..., b]
    y[..., a] = x1 * cos - x2 * sin
    y[..., b] = x2 * cos + x1 * sin
    return y


def _grid(s):
    """Which rows of the batch each sequence's new tokens are: [seqs, queries], and whether they exist."""
    at = torch.arange(s["queries"], device="cuda")
    if s["starts"] is None:
        return torch.arange(s["seqs"], device="cuda")[:, None], torch.ones(s["seqs"], 1, dtype=torch.bool, device="cuda")
    first, new = s["starts"][:-1].long(), s["starts"].diff().long()
    return (first[:, None] + at).clamp(max=s["q"].shape[0] - 1), at < new[:, None]


def _new(s):
    return torch.ones_like(s["lengths"]).long() if s["starts"] is None else s["starts"].diff().long()


def _sequence_of(s, rows):
    """Each row's sequence and place among its new tokens."""
    row = torch.arange(rows, device="cuda")
    if s["starts"] is None:
        return row, torch.zeros_like(row)
    b = torch.searchsorted(s["starts"], row.int(), right=True) - 1
    return b, row - s["starts"][b]


def _append(s):
    block, page, fmt, pairs = s["block"], s["page"], s["fmt"], s["pairs"]
    length, new = s["lengths"].long(), _new(s)
    b, i = _sequence_of(s, s["q"].shape[0])
    position = length[b] - new[b] + i
    cos, sin = s["cos"][position][:, None], s["sin"][position][:, None]
    k = _rotate(s["new_k"].float(), cos, sin, pairs, s["interleaved"])
    q = _rotate(s["q"].float(), cos, sin, pairs, s["interleaved"])
    # the blocks that get new tokens: [seqs, blocks, block] positions, each sequence's from its first such block on
    held = length - new
    blocks = (s["queries"] + block - 2) // block + 1
    at = (held // block * block)[:, None, None] + torch.arange(blocks * block, device="cuda").reshape(blocks, block)
    is_new = (at >= held[:, None, None]) & (at < length[:, None, None])
    is_held = at < held[:, None, None]
    touched = is_new.any(-1, keepdim=True)
    first = torch.arange(s["seqs"], device="cuda") if s["starts"] is None else s["starts"][:-1].long()
    row = ((first - held)[:, None, None] + at).clamp(0, s["q"].shape[0] - 1)
    to = torch.gather(s["table"].long(), 1, (at // page).flatten(1)).reshape(at.shape)
    slot, part = at % page, at[..., 0] % page // block
    for x, (codes, scales) in ((k, s["k"]), (s["new_v"].float(), s["v"])):
        x = torch.where(is_new[..., None, None], x[row], 0.0)            # [seqs, blocks, block, heads, dim]
        old = scales[to[..., 0], :, part]                                # [seqs, blocks, heads]
        was = torch.where(is_held.any(-1)[..., None], old, 0.0)
        # (a division by a number would be a product with its rounded reciprocal)
        scale = torch.maximum(was, x.abs().amax((2, 4)) / torch.full((), QMAX[fmt], device="cuda"))
        safe = torch.where(scale > 0, scale, 1.0)
        c = codes[to, :, slot]                                           # [seqs, blocks, block, heads, dim]
        again = _round_codes(c.view(VIEW[fmt]).float() * (was / safe)[:, :, None, :, None], fmt)
        fresh = _round_codes(x / safe[:, :, None, :, None], fmt)
        c = torch.where(is_new[..., None, None], fresh, torch.where((is_held & touched)[..., None, None], again, c))
        codes[to, :, slot] = c
        scales[to[..., 0], :, part] = torch.where(touched, scale, old)
    return _contents(s, q.to(s["q"].dtype))


def _gathered(s, codes, scales):
    """[seqs, heads, tokens, dim] of the cache's values, fp32."""
    n, heads, page, dim = codes.shape
    x = codes[s["table"].long()].view(VIEW[s["fmt"]]).float()            # [seqs, pages, heads, page, dim]
    x = x.reshape(*x.shape[:3], page // s["block"], s["block"], dim) * scales[s["table"].long()][..., None, None]
    return x.permute(0, 2, 1, 3, 4, 5).reshape(s["seqs"], heads, -1, dim)


def _attention(s):
    heads, kv, dim, most = s["heads"], s["kv_heads"], s["dim"], s["queries"]
    rows, _ = _grid(s)
    q = s["q"].float()[rows].reshape(s["seqs"], -1, kv, heads // kv, dim).permute(0, 2, 1, 3, 4).reshape(s["seqs"], kv, -1, dim)
    k = _gathered(s, *s["k"])
    score = q @ k.transpose(-1, -2) / math.sqrt(dim)                     # [seqs, kv, queries x group, tokens]
    del k
    at = torch.arange(score.shape[-1], device="cuda")
    last = (s["lengths"].long() - _new(s))[:, None] + torch.arange(rows.shape[1], device="cuda")
    seen = (at <= last[..., None]) & (at < s["lengths"][:, None, None])
    if s["window"]:
        seen &= at > last[..., None] - s["window"]
    seen = seen[:, None, :, None].expand(-1, -1, -1, heads // kv, -1).flatten(2, 3)
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = p @ _gathered(s, *s["v"]) / torch.where(total > 0, total, 1.0)
    lse = (total.log() + top)[..., 0]
    b, i = _sequence_of(s, s["q"].shape[0])
    out = out.reshape(s["seqs"], kv, -1, heads // kv, dim)[b, :, i].reshape(-1, heads, dim).to(torch.bfloat16)
    return (out, lse.reshape(s["seqs"], kv, -1, heads // kv)[b, :, i].reshape(-1, heads)) if s["lse"] else out


def run(s):
    if own:
        return _run_own(s)
    if s["op"].startswith("rotary"):
        cos, sin = s["cos"][s["positions"]][:, None], s["sin"][s["positions"]][:, None]
        if s["op"] == "rotary_backward":
            sin = -sin
        return _rotate(s["x"].float(), cos, sin, s["pairs"], s["interleaved"]).to(s["x"].dtype)
    return _append(s) if s["op"] == "append" else _attention(s)


def work(case):
    op, dim = case["op"], case["dim"]
    e = 4 if case.get("dtype") == "f32" else 2
    if op.startswith("rotary"):
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * dim * e + case["tokens"] * (8 * case["pairs"] + 4), "flops": 6 * n * case["pairs"]}
    length, new = _lengths(case)
    heads, kv, block, tokens = case["heads"], case["kv_heads"], case["block"], sum(new)
    if op == "append":
        blocks = sum(-(-n // block) - (n - m) // block for n, m in zip(length, new))
        held = sum((n - m) % block for n, m in zip(length, new))
        values = tokens * dim * (heads + 2 * kv)
        return {"bytes": tokens * (e * dim * (2 * heads + 2 * kv) + 2 * kv * dim + 8 * case["pairs"]) + 2 * kv * (8 * blocks + held * dim),
                "flops": 8 * values}
    first = [max(0, n - m + 1 - case["window"]) if case["window"] else 0 for n, m in zip(length, new)]
    read = sum(n - f for n, f in zip(length, first))
    pairs = 0
    for n, m in zip(length, new):
        if case["window"]:
            pairs += sum(min(case["window"], n - m + i + 1) for i in range(m))
        else:
            pairs += m * (n - m) + m * (m + 1) // 2
    return {"bytes": 2 * kv * read * (dim + 4 / block) + tokens * heads * (4 * dim + (4 if case["lse"] else 0)), "flops": 4 * dim * heads * pairs}


# ---- the definition in 64 bits ------------------------------------------------------------------
def _turn64(x, position, cos, sin, pairs, interleaved, back=False):
    """Each pair as a complex number times cos + i sin, or its conjugate."""
    x, z = x.double().clone(), torch.complex(cos.double(), sin.double())[position.long()][:, None]
    if back:
        z = z.conj()
    if interleaved:
        w = torch.view_as_complex(x[..., :2 * pairs].reshape(*x.shape[:-1], pairs, 2)) * z
        x[..., :2 * pairs] = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(x[..., :pairs].contiguous(), x[..., pairs:2 * pairs].contiguous()) * z
        x[..., :2 * pairs] = torch.cat((w.real, w.imag), -1)
    return x


def _value64(codes, fmt):
    """The numbers that the codes stand for, from their fields."""
    c = codes.to(torch.int64)
    if fmt == "int8":
        return torch.where(c > 127, c - 256, c).double()
    m = 3 if fmt == "e4m3" else 2
    bias, e, f = (7 if m == 3 else 15), (c & 127) >> m, (c & ((1 << m) - 1)).double() / (1 << m)
    v = torch.where(e > 0, torch.ldexp(1 + f, (e - bias).double()), torch.ldexp(f, torch.full_like(f, 1.0 - bias)))
    return torch.where(c > 127, -v, v)


def _nearest64(v, fmt):
    """The format's number nearest to v, ties to the even one."""
    v = v.clamp(-QMAX[fmt], QMAX[fmt])
    if fmt == "int8":
        return v.round()
    m, least = (3, -6) if fmt == "e4m3" else (2, -14)
    e = torch.frexp(v.abs()).exponent.double() - 1
    step = torch.exp2(e.clamp(min=least) - m)
    return (v / step).round() * step


def _append64(s, length, new):
    block, page, fmt = s["block"], s["page"], s["fmt"]
    values = {}
    q_out, row = [], 0
    for name in ("k", "v"):
        codes, scales = s[name]
        values[name] = [_value64(codes, fmt), scales.double()]
    for b, (n, m) in enumerate(zip(length, new)):
        position = torch.arange(n - m, n, device="cuda")
        turn = (position, s["cos"], s["sin"], s["pairs"], s["interleaved"])
        q_out.append(_turn64(s["q"][row:row + m], *turn))
        k = _turn64(s["new_k"][row:row + m], *turn)
        row += m
        for name, x in (("k", k), ("v", s["new_v"][row - m:row].double())):
            value, scale = values[name]
            first, heads = (n - m) // block, x.shape[1]
            held, blocks = (n - m) - first * block, -(-n // block) - first
            whole = torch.zeros(blocks * block, heads, x.shape[2], dtype=torch.float64, device="cuda")
            whole[held:held + m] = x
            whole = whole.reshape(blocks, block, heads, -1)
            j = torch.arange(first, first + blocks, device="cuda")
            at = s["table"][b, j * block // page].long(), slice(None), j * block % page // block
            old = scale[at].clone()
            if held == 0:
                old[0] = 0
            old[1:] = 0
            now = torch.maximum(old, whole.abs().amax((1, 3)) / QMAX[fmt])
            scale[at] = now
            now = torch.where(now > 0, now, 1.0)
            p = torch.arange(first * block, n, device="cuda")
            where = s["table"][b, p // page].long(), slice(None), p % page
            kept = value[where]
            fresh = _nearest64(whole / now[:, None, :, None], fmt).reshape(blocks * block, heads, -1)[:held + m]
            fresh[:held] = _nearest64(kept[:held] * (old[0] / now[0])[:, None], fmt)
            value[where] = fresh
    codes = [None if fmt == "int8" else values[name][0] for name in ("k", "v")]
    return torch.cat(q_out), codes[0], values["k"][1], codes[1], values["v"][1]


def exact(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if op.startswith("rotary"):
        return _turn64(s["x"], s["positions"], s["cos"], s["sin"], case["pairs"], case["interleaved"], op == "rotary_backward")
    length, new = _lengths(case)
    if op == "append":
        return _append64(s, length, new)
    kv, group, page, block = case["kv_heads"], case["heads"] // case["kv_heads"], case["page"], case["block"]
    out = torch.zeros(sum(new), case["heads"], case["dim"], dtype=torch.float64, device="cuda")
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, m) in enumerate(zip(length, new)):
        p = torch.arange(n, device="cuda")
        at = s["table"][b, p // page].long()
        last = torch.arange(n - m, n, device="cuda")
        hidden = p > last[:, None]
        if case["window"]:
            hidden |= p <= last[:, None] - case["window"]
        for h in range(kv):
            k, v = (_value64(c[at, h, p % page], case["fmt"]) * z[at, h, p % page // block].double()[:, None] for c, z in (s["k"], s["v"]))
            for g in range(h * group, (h + 1) * group):
                t = torch.einsum("td,nd->tn", s["q"][row:row + m, g].double(), k).div_(case["dim"] ** 0.5)
                t.masked_fill_(hidden, -math.inf)
                lse[row:row + m, g] = torch.logsumexp(t, -1)
                out[row:row + m, g] = torch.einsum("tn,nd->td", torch.softmax(t, -1), v)
        row += m
    return (out, lse) if case["lse"] else out
