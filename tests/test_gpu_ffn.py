"""Products with 4-bit weights and the gated block on the GPU, against 64-bit references."""
import numpy as np
import pytest

import ffn_util as F

pytestmark = pytest.mark.gpu

# (tokens, rows, cols): one token, odd outputs, a ragged last tile along every axis, sums that
# end inside a 64-wide step, more tokens than one tile
SHAPES = [(1, 1, 128), (1, 1000, 4096), (2, 77, 384), (3, 16, 640), (5, 129, 256), (8, 520, 2048),
          (9, 300, 512), (16, 264, 1152), (33, 1023, 384), (65, 128, 896), (130, 513, 1280),
          (257, 328, 640), (300, 640, 4224), (513, 264, 256)]


@pytest.fixture(scope="module")
def qz():
    import __graft_entry__
    __graft_entry__.build_library()
    import precision_quantization_gb300 as qz
    qz.lib()
    return qz


def check_linear(qz, w, x, out="bf16", **view):
    import torch
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    got = F.host(qz.linear(F.bf16_cuda(x, **view), F.handle(w), out_dtype=dt))
    want = x @ w["values"].T
    bound = F.sum_bound(x.shape[1], np.abs(x) @ np.abs(w["values"]).T)
    F.assert_within(got, want, bound * 1.01 + (F.bf16_bound(want) if out == "bf16" else 0))
    return got


@pytest.mark.parametrize("fmt", list(F.FORMATS))
@pytest.mark.parametrize("shape", SHAPES)
def test_linear(qz, fmt, shape):
    rng = np.random.default_rng(hash(shape) % 1000)
    w = F.make_weight(rng, fmt, *shape[1:])
    x = F.activations(rng, shape[0], shape[2])
    check_linear(qz, w, x, "bf16")
    check_linear(qz, w, x, "f32")


@pytest.mark.parametrize("fmt", list(F.FORMATS))
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_exact(qz, fmt, shape):
    """Small integers and power-of-two scales: every partial sum is exact in fp32, so a dropped,
    doubled or misplaced term shows whatever the order of the sum."""
    import torch
    rng = np.random.default_rng(hash(shape) % 1000 + 1)
    w = F.make_weight(rng, fmt, *shape[1:], exact=True)
    x = F.activations(rng, shape[0], shape[2], exact=True)
    h = F.handle(w)
    got = F.host(qz.linear(F.bf16_cuda(x), h, out_dtype=torch.float32))
    assert np.array_equal(got, x @ w["values"].T)
    dy = F.activations(rng, shape[0], shape[1], exact=True)
    got = F.host(qz.linear_backward(F.bf16_cuda(dy), h, out_dtype=torch.float32))
    assert np.array_equal(got, dy @ w["values"])


@pytest.mark.parametrize("group", [16, 32, 64, 128])
@pytest.mark.parametrize("tokens", [1, 6, 40, 200])
def test_int4_groups(qz, group, tokens):
    import torch
    rng = np.random.default_rng(group + tokens)
    w = F.make_weight(rng, "int4", 200, 5 * 128, group)
    x = F.activations(rng, tokens, 640)
    check_linear(qz, w, x, "f32")
    dy = F.activations(rng, tokens, 200)
    got = F.host(qz.linear_backward(F.bf16_cuda(dy), F.handle(w), out_dtype=torch.float32))
    F.assert_within(got, dy @ w["values"], F.sum_bound(200, np.abs(dy) @ np.abs(w["values"])))


# sums that are no multiple of 32 (16-wide blocks), and views whose rows are not 16-byte aligned
@pytest.mark.parametrize("tokens", [1, 7, 100])
@pytest.mark.parametrize("view", [dict(), dict(pad=8), dict(pad=3), dict(lead=1, pad=7), dict(lead=8)])
@pytest.mark.parametrize("cols", [48, 64, 2064])
def test_linear_strides(qz, tokens, view, cols):
    rng = np.random.default_rng(cols + tokens)
    w = F.make_weight(rng, "nvfp4", 70, cols)
    check_linear(qz, w, F.activations(rng, tokens, cols), **view)


@pytest.mark.parametrize("tokens", [8, 9, 10, 15, 16, 17])
@pytest.mark.parametrize("cols", [8192, 9088])
def test_int4_tokens_in_two_halves(qz, tokens, cols):
    """Activations too large for one CTA's shared memory, next to ones that still fit."""
    import torch
    rng = np.random.default_rng(tokens + cols)
    w = F.make_weight(rng, "int4", 45, cols, 64, exact=True)
    x = F.activations(rng, tokens, cols, exact=True)
    h, want = F.handle(w), x @ w["values"].T
    for dt, pad in ((torch.float32, 0), (torch.bfloat16, 3)):
        buf = torch.full((tokens, 45 + pad), 7.0, dtype=dt, device="cuda")
        qz.linear(F.bf16_cuda(x, pad=8), h, out=buf[:, :45])
        assert np.all(np.abs(F.host(buf[:, :45]) - want) <= (F.bf16_bound(want) if dt == torch.bfloat16 else 0))
        assert bool((buf[:, 45:] == 7).all())
    _, g, u = qz.gated_ffn(F.bf16_cuda(x), h, h, save=True)
    assert np.array_equal(F.host(g), F.host(u)) and np.all(np.abs(F.host(g) - want) <= F.bf16_bound(want))


@pytest.mark.parametrize("offset", [0, 1, 2])
@pytest.mark.parametrize("fmt,group", [("mxfp4", 32), ("nvfp4", 16), ("int4", 32), ("int4", 64), ("int4", 128)])
@pytest.mark.parametrize("shape", [(1, 33, 32), (1, 50, 224), (4, 1003, 288), (6, 16, 992), (11, 40, 1376), (20, 70, 544),
                                   (32, 31, 96), (27, 300, 4064)])
def test_linear_narrow_rows(qz, fmt, group, shape, offset):
    """Up to 32 tokens with rows that are not whole 256-column steps, and scales at odd places."""
    import torch
    tokens, rows, cols = shape[0], shape[1], -(-shape[2] // group) * group
    rng = np.random.default_rng(hash(shape) % 1000 + group)
    w = F.make_weight(rng, fmt, rows, cols, group, exact=True)
    x = F.activations(rng, tokens, cols, exact=True)
    h = F.handle(w)
    if offset:
        s = h.q.scales.reshape(-1)
        buf = torch.zeros(s.numel() + offset, dtype=s.dtype, device="cuda")
        buf[offset:] = s
        h.q.scales = buf[offset:].reshape(h.q.scales.shape)
        h = qz.Weight(h.q)
    got = F.host(qz.linear(F.bf16_cuda(x), h, out_dtype=torch.float32))
    assert np.array_equal(got, x @ w["values"].T)
    if not offset:
        check_linear(qz, F.make_weight(rng, fmt, rows, cols, group), F.activations(rng, tokens, cols), "f32")
        up = F.handle(w)
        hid, g, u = qz.gated_ffn(F.bf16_cuda(x), h, up, save=True)
        assert np.array_equal(F.host(g), F.host(u))
        assert np.all(np.abs(F.host(g) - x @ w["values"].T) <= F.bf16_bound(x @ w["values"].T))


@pytest.mark.parametrize("tokens", [1, 5, 70])
def test_linear_codes_offset(qz, tokens):
    """Codes that start at an odd byte, and an output view inside a larger tensor."""
    import torch
    rng = np.random.default_rng(tokens)
    w = F.make_weight(rng, "mxfp4", 96, 256)
    x = F.activations(rng, tokens, 256)
    h = F.handle(w)
    buf = torch.zeros(96 * 128 + 1, dtype=torch.uint8, device="cuda")
    buf[1:] = h.q.codes.reshape(-1)
    h.q.codes = buf[1:].reshape(96, 128)
    h = qz.Weight(h.q)
    big = torch.full((tokens, 131), 7.0, dtype=torch.bfloat16, device="cuda")
    qz.linear(F.bf16_cuda(x), h, out=big[:, 5:101])
    want = x @ w["values"].T
    F.assert_within(F.host(big[:, 5:101]), want,
                    F.bf16_bound(want) + F.sum_bound(256, np.abs(x) @ np.abs(w["values"]).T))
    assert bool((big[:, :5] == 7).all()) and bool((big[:, 101:] == 7).all())


@pytest.mark.parametrize("tokens", [1, 8, 50, 300])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_scale_range(qz, fmt, tokens):
    """Block scales at the ends of their range: 2^-127 .. 2^127 and the E4M3 subnormals."""
    import torch
    rng = np.random.default_rng(tokens)
    w = F.make_weight(rng, fmt, 64, 256)
    if fmt == "mxfp4":
        lo, x_scale = ([-127, -126, -125, -100], 2.0 ** 100) if tokens % 2 else ([100, 110, 120, 1], 2.0 ** -60)
        k = np.array(lo)[rng.integers(0, 4, (64, 8))]
        w["scales"] = (k + 127).astype(np.uint8)
        w["values"] = w["elements"] * np.repeat(np.ldexp(1.0, k), 32, axis=1)
    else:
        x_scale = 1.0
        s = np.array([0x00, 0x01, 0x07, 0x08, 0x7E])[rng.integers(0, 5, (64, 16))]
        w["scales"] = s.astype(np.uint8)
        w["values"] = w["elements"] * np.repeat(F.e4m3_value(s) * np.float64(w["ts"]), 16, axis=1)
    x = F.activations(rng, tokens, 256) * x_scale
    got = F.host(qz.linear(F.bf16_cuda(x), F.handle(w), out_dtype=torch.float32))
    F.assert_within(got, x @ w["values"].T, F.sum_bound(256, np.abs(x) @ np.abs(w["values"]).T))


@pytest.mark.parametrize("tokens", [1, 4, 60, 200])
@pytest.mark.parametrize("fmt", list(F.FORMATS))
def test_nonfinite_stays_in_its_token(qz, fmt, tokens):
    rng = np.random.default_rng(3)
    w = F.make_weight(rng, fmt, 150, 384)
    x = F.activations(rng, tokens, 384)
    h = F.handle(w)
    clean = F.host(qz.linear(F.bf16_cuda(x), h))
    bad = x.copy()
    bad[0, 5] = np.nan
    if tokens > 2:
        bad[2, 300] = np.inf
    got = F.host(qz.linear(F.bf16_cuda(bad), h))
    assert np.isnan(got[0]).all()
    if tokens > 2:
        v = w["values"][:, 300]
        assert np.isnan(got[2][v == 0]).all()
        if fmt == "int4":  # a weight may be held as two terms, whose products with Inf need not agree
            assert not np.isfinite(got[2][v != 0]).any()
        else:
            assert np.array_equal(got[2][v != 0], np.sign(v[v != 0]) * np.inf)
    keep = [t for t in range(tokens) if t not in (0, 2)] if tokens > 2 else list(range(1, tokens))
    assert np.array_equal(got[keep], clean[keep])


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_same_inputs_same_bits_on_any_stream(qz, tokens):
    import torch
    rng = np.random.default_rng(tokens)
    w = F.make_weight(rng, "nvfp4", 1000, 2048)
    x, h = F.bf16_cuda(F.activations(rng, tokens, 2048)), F.handle(w)
    a = qz.linear(x, h, out_dtype=torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = qz.linear(x, h, out_dtype=torch.float32)
    c = qz.linear(x, h, out_dtype=torch.float32, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


def test_empty(qz):
    import torch
    rng = np.random.default_rng(0)
    h = F.handle(F.make_weight(rng, "mxfp4", 64, 128))
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    assert qz.linear(x, h).shape == (0, 64)
    assert qz.gated_ffn(x, h, h).shape == (0, 64)
    dh = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert qz.linear_backward(dh, h).shape == (0, 128)
    assert [t.shape for t in qz.gated_ffn_backward(dh, dh, dh, h, h)] == [(0, 128), (0, 64), (0, 64)]
    none = F.handle(dict(F.make_weight(rng, "int4", 8, 128), codes=np.zeros((8, 0), np.uint8),
                         scales=np.zeros((8, 0), np.float32), cols=0))
    z = qz.linear(torch.empty((3, 0), dtype=torch.bfloat16, device="cuda"), none)
    assert z.shape == (3, 8) and bool((z == 0).all())  # empty sums


@pytest.mark.parametrize("fmt", list(F.FORMATS))
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_backward(qz, fmt, shape):
    tokens, rows, cols = shape
    rng = np.random.default_rng(rows)
    w = F.make_weight(rng, fmt, rows, cols)
    dy = F.activations(rng, tokens, rows, scale=0.01)
    got = F.host(qz.linear_backward(F.bf16_cuda(dy), F.handle(w)))
    want = dy @ w["values"]
    F.assert_within(got, want, F.bf16_bound(want) + F.sum_bound(rows, np.abs(dy) @ np.abs(w["values"])) * 1.01)


@pytest.mark.parametrize("tokens", [1, 8, 90])
def test_linear_backward_is_the_forward_difference(qz, tokens):
    """<dy, f(x + d) - f(x)> = <dx, d>: f is linear, the steps are exact bf16 values."""
    import torch
    rng = np.random.default_rng(tokens)
    w = F.make_weight(rng, "nvfp4", 256, 512)
    h = F.handle(w)
    x, d = F.activations(rng, tokens, 512, exact=True), rng.integers(-3, 4, (tokens, 512)).astype(np.float64)
    dy = F.activations(rng, tokens, 256)
    f = lambda a: F.host(qz.linear(F.bf16_cuda(a), h, out_dtype=torch.float32))  # noqa: E731
    dx = F.host(qz.linear_backward(F.bf16_cuda(dy), h, out_dtype=torch.float32))
    left, right = (dy * (f(x + d) - f(x))).sum(), (dx * d).sum()
    a = np.abs(w["values"])
    room = (np.abs(dy) * F.sum_bound(512, (2 * np.abs(x) + np.abs(d)) @ a.T)).sum() + \
        (np.abs(d) * F.sum_bound(256, np.abs(dy) @ a)).sum()
    assert abs(left - right) <= room


GATED = [(1, 8, 128), (1, 1000, 2048), (4, 72, 512), (8, 200, 640), (17, 136, 256), (64, 1000, 384),
         (129, 264, 640), (300, 520, 1024), (513, 64, 256)]


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("fmt", list(F.FORMATS))
@pytest.mark.parametrize("shape", GATED)
def test_gated(qz, kind, fmt, shape):
    tokens, rows, cols = shape
    rng = np.random.default_rng(rows + cols)
    wg, wu = (F.make_weight(rng, fmt, rows, cols) for _ in range(2))
    x = F.activations(rng, tokens, cols)
    xt, gate, up = F.bf16_cuda(x), F.handle(wg), F.handle(wu)
    h, g, u = qz.gated_ffn(xt, gate, up, activation=kind, save=True)
    gw, uw = x @ wg["values"].T, x @ wu["values"].T
    gb, ub = (F.sum_bound(cols, np.abs(x) @ np.abs(w["values"]).T) for w in (wg, wu))
    F.assert_within(F.host(g), gw, gb + F.bf16_bound(gw), "g")
    F.assert_within(F.host(u), uw, ub + F.bf16_bound(uw), "u")
    # h = a(g) u: |a'| <= 1.2 moves g's error, |a(g)| <= |g| + 0.2 takes u's; 2^-18 of the product
    # covers the activation's own fp32 evaluation (its exponential has a few ulp)
    a = F.act(gw, kind)[0]
    bound = 1.2 * gb * (np.abs(uw) + ub) + np.abs(a) * ub + 2.0 ** -18 * (np.abs(gw) + 1) * np.abs(uw)
    F.assert_within(F.host(h), a * uw, bound + F.bf16_bound(a * uw), "h")
    assert np.array_equal(F.host(qz.gated_ffn(xt, gate, up, activation=kind)), F.host(h))


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("fmt", list(F.FORMATS))
@pytest.mark.parametrize("shape", GATED)
def test_gated_backward(qz, kind, fmt, shape):
    tokens, rows, cols = shape
    rng = np.random.default_rng(rows * 3 + cols)
    wg, wu = (F.make_weight(rng, fmt, rows, cols) for _ in range(2))
    dh = F.activations(rng, tokens, rows, scale=0.1)
    g, u = (F.activations(rng, tokens, rows, scale=3.0) for _ in range(2))
    dx, dg, du = qz.gated_ffn_backward(F.bf16_cuda(dh), F.bf16_cuda(g), F.bf16_cuda(u), F.handle(wg), F.handle(wu),
                                       activation=kind)
    a, da = F.act(g, kind)
    # the activation and its derivative are evaluated in fp32 with an absolute error of a few
    # ulp of (1 + |g|^2): both are sums of terms no larger than that
    slack = 2.0 ** -18 * (1 + g * g) * np.abs(dh)
    F.assert_within(F.host(dg), dh * u * da, F.bf16_bound(dh * u * da) + slack * np.abs(u), "dg")
    F.assert_within(F.host(du), dh * a, F.bf16_bound(dh * a) + slack, "du")
    # dx is the product of the rounded dg and du, which the call returns
    rg, ru = F.host(dg), F.host(du)
    want = rg @ wg["values"] + ru @ wu["values"]
    terms = np.abs(rg) @ np.abs(wg["values"]) + np.abs(ru) @ np.abs(wu["values"])
    F.assert_within(F.host(dx), want, F.bf16_bound(want) + F.sum_bound(2 * rows, terms), "dx")


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gated_gradient_is_the_difference(qz, kind):
    """The gradient of sum(dh * h) along a direction, against central differences of the block
    itself in 64 bits about the same kept pre-activations."""
    rng = np.random.default_rng(8)
    wg, wu = (F.make_weight(rng, "mxfp4", 96, 128) for _ in range(2))
    x, dh = F.activations(rng, 5, 128, scale=0.3), F.activations(rng, 5, 96)
    d = rng.normal(size=x.shape)
    f = lambda v: (dh * F.act(v @ wg["values"].T, kind)[0] * (v @ wu["values"].T)).sum()  # noqa: E731
    slope = (f(x + 1e-5 * d) - f(x - 1e-5 * d)) / 2e-5
    _, g, u = qz.gated_ffn(F.bf16_cuda(x), F.handle(wg), F.handle(wu), activation=kind, save=True)
    dx, _, _ = qz.gated_ffn_backward(F.bf16_cuda(dh), g, u, F.handle(wg), F.handle(wu), activation=kind)
    # g, u, dg, du and dx are each rounded to bf16 (2^-9 relative, independent): their effect on
    # the sum stays under five times 2^-9 of the sum of the terms' magnitudes
    a, da = F.act(x @ wg["values"].T, kind)
    mag = (np.abs(d) * ((np.abs(dh * (x @ wu["values"].T)) * 1.2) @ np.abs(wg["values"]) +
                        (np.abs(dh) * (np.abs(a) + 1.2)) @ np.abs(wu["values"]))).sum()
    assert abs((F.host(dx) * d).sum() - slope) <= 5 * 2.0 ** -9 * mag


def test_gated_limits(qz):
    """Pre-activations at +-inf and far out: the limits of the activation, not NaN."""
    import torch
    rng = np.random.default_rng(1)
    w = F.handle(F.make_weight(rng, "mxfp4", 8, 32))
    g = np.array([[-np.inf, np.inf, -3e38, 3e38, -200.0, 200.0, 0.0, -0.0]])
    one = np.ones_like(g)
    for kind in ("silu", "gelu_tanh"):
        _, dg, du = qz.gated_ffn_backward(F.bf16_cuda(one), F.bf16_cuda(g), F.bf16_cuda(one), w, w, activation=kind)
        assert np.array_equal(F.host(dg)[0], [0, 1, 0, 1, 0, 1, 0.5, 0.5])
        want = F.bf16_cuda(np.array([[0, np.inf, 0, 3e38, 0, 200.0, 0, 0]])).float().cpu()
        assert torch.equal(du.float().cpu().abs(), want)


@pytest.mark.parametrize("view", [dict(pad=3), dict(pad=8)])
@pytest.mark.parametrize("tokens", [3, 150])
def test_gated_strides(qz, view, tokens):
    import torch
    rng = np.random.default_rng(5)
    wg, wu = (F.make_weight(rng, "nvfp4", 104, 192) for _ in range(2))
    gate, up = F.handle(wg), F.handle(wu)
    x, dh = F.activations(rng, tokens, 192), F.activations(rng, tokens, 104)
    outs = [torch.full((tokens, 104 + view["pad"]), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    h, g, u = qz.gated_ffn(F.bf16_cuda(x, **view), gate, up, save=True, out=[o[:, :104] for o in outs])
    plain = qz.gated_ffn(F.bf16_cuda(x), gate, up, save=True)
    bound = F.sum_bound(192, np.abs(x) @ np.abs(wg["values"]).T)
    for a, b in zip((h, g, u), plain):
        rows_b = 30 * bound * (1 + np.abs(F.host(b))) + 2 * F.bf16_bound(F.host(b))
        F.assert_within(F.host(a), F.host(b), rows_b)
    for o in outs:
        assert bool((o[:, 104:] == 9).all())
    gs, us, ds = (F.bf16_cuda(F.host(t), **view) for t in (g, u, F.bf16_cuda(dh)))
    dx, dg, du = qz.gated_ffn_backward(ds, gs, us, gate, up)
    dx2, dg2, du2 = qz.gated_ffn_backward(F.bf16_cuda(dh), g.contiguous(), u.contiguous(), gate, up)
    assert torch.equal(dg, dg2) and torch.equal(du, du2) and torch.equal(dx, dx2)
