"""The forms that the products with 4-bit weights take by size: exact integer sums, so that a dropped,
doubled or misplaced term shows whatever the order of the sum."""
import numpy as np
import pytest

import ffn_util as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qz():
    import __graft_entry__
    __graft_entry__.build_library()
    import precision_quantization_gb300 as qz
    qz.lib()
    return qz


@pytest.mark.parametrize("ld", [1 << 20, (1 << 40) + 8, (1 << 41) + 3])
@pytest.mark.parametrize("fmt", list(F.FORMATS))
def test_one_token_has_any_leading_dimension(qz, fmt, ld):
    """One row is one row, whatever its leading dimension: no second one is ever addressed."""
    import torch
    rng = np.random.default_rng(4)
    w = F.make_weight(rng, fmt, 72, 256, exact=True)
    h = F.handle(w)
    x, dy = F.activations(rng, 1, 256, exact=True), F.activations(rng, 1, 72, exact=True)
    xt, dyt, y, dx = F.bf16_cuda(x), F.bf16_cuda(dy), torch.empty(72, device="cuda"), torch.empty(256, device="cuda")
    assert qz.qz_linear(h.desc, xt.data_ptr(), ld, 1, y.data_ptr(), ld, qz.QZ_F32) == qz.QZ_OK
    assert qz.qz_linear_backward(h.desc, dyt.data_ptr(), ld, 1, dx.data_ptr(), ld, qz.QZ_F32) == qz.QZ_OK
    torch.cuda.synchronize()
    assert np.array_equal(F.host(y), (x @ w["values"].T)[0]) and np.array_equal(F.host(dx), (dy @ w["values"])[0])
    want = qz.gated_ffn(xt, h, h, save=True)
    got = [torch.empty(72, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    p = [t.data_ptr() for t in got]
    assert qz.qz_gated_ffn(h.desc, h.desc, qz.QZ_ACT_SILU, xt.data_ptr(), ld, 1, p[0], ld, p[1], p[2], ld) == qz.QZ_OK
    torch.cuda.synchronize()
    assert all(torch.equal(a, b[0]) for a, b in zip(got, want))
    wdx, wdg, wdu = qz.gated_ffn_backward(dyt, want[1], want[2], h, h)
    gdx = torch.empty(256, dtype=torch.bfloat16, device="cuda")
    assert qz.qz_gated_ffn_backward(h.desc, h.desc, qz.QZ_ACT_SILU, dyt.data_ptr(), ld, want[1].data_ptr(), want[2].data_ptr(),
                                    ld, 1, p[0], p[1], ld, gdx.data_ptr(), ld) == qz.QZ_OK
    torch.cuda.synchronize()
    assert torch.equal(gdx, wdx[0]) and torch.equal(got[0], wdg[0]) and torch.equal(got[1], wdu[0])


# The forms below are those that the launch plan takes on 152 SMs.  (mode, tokens, outputs, summands):
# pairs of CTAs with three tiles and more each (both accumulators come round again, decoders run on
# into the next tile), tiles of 64, 192 and 256 tokens, one and several of them a row
PAIRS = [(33, 60000, 128), (250, 60000, 160), (513, 20000, 128), (700, 20000, 96)]
# a second launch for the outputs that would start a nearly empty round: linear, gated, backward, both weights'
TWO_E2M1 = [("linear", 131, 20008, 4096), ("gated", 250, 10024, 2048), ("backward", 131, 20000, 4096), ("both", 33, 20000, 2048)]
TWO_INT4 = [("linear", 77, 20008, 1152), ("gated", 33, 10024, 1152), ("backward", 77, 20000, 1152), ("both", 33, 20000, 640)]
# the streaming kernel: several tiles at once in a CTA (over 2432 outputs), and several rounds of them
FEW = [(1, 5003, 128), (5, 41003, 128), (16, 41003, 288), (9, 5003, 4352)]


def double(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().double()


def pair(fmt, rows, cols, seed, **k):
    rng = np.random.default_rng(seed)
    w = F.make_weight(rng, fmt, rows, cols, **k)
    return rng, w, double(w["values"])


def linear_exactly(qz, fmt, tokens, rows, cols, group=None):
    import torch
    rng, w, v = pair(fmt, rows, cols, tokens + cols, exact=True, group=group)
    x = F.activations(rng, tokens, cols, exact=True)
    xt, h, want = F.bf16_cuda(x), F.handle(w), double(x) @ v.T
    assert torch.equal(qz.linear(xt, h, out_dtype=torch.float32).double(), want)
    assert torch.equal(qz.linear(xt, h), want.to(torch.float32).to(torch.bfloat16))  # one rounding


def backward_exactly(qz, fmt, tokens, cols, rows):
    import torch
    rng, w, v = pair(fmt, rows, cols, tokens + rows, exact=True)
    dy = F.activations(rng, tokens, rows, exact=True)
    got = qz.linear_backward(F.bf16_cuda(dy), F.handle(w), out_dtype=torch.float32)
    assert torch.equal(got.double(), double(dy) @ v)


def gated_exactly(qz, fmt, tokens, rows, cols):
    import torch
    rng, wg, vg = pair(fmt, rows, cols, tokens + cols, exact=True)
    _, wu, vu = pair(fmt, rows, cols, tokens + cols + 1, exact=True)
    x = F.activations(rng, tokens, cols, exact=True)
    h, g, u = qz.gated_ffn(F.bf16_cuda(x), F.handle(wg), F.handle(wu), save=True)
    gw, uw = double(x) @ vg.T, double(x) @ vu.T
    bf = lambda t: t.to(torch.float32).to(torch.bfloat16)  # noqa: E731
    assert torch.equal(g, bf(gw)) and torch.equal(u, bf(uw))
    # the activation in fp32 (2^-18 of |g| + 1, as for exact sums elsewhere), and one rounding to bf16
    want = gw * torch.sigmoid(gw) * uw
    assert bool(((h.double() - want).abs() <= 2.0 ** -18 * (gw.abs() + 1) * uw.abs() + 2.0 ** -8 * 1.01 * want.abs()).all())


def both_backward(qz, fmt, tokens, cols, rows):
    """dx of the gated block: integers for dg and du would need g and u that give them, so the sum's bound."""
    rng, wg, vg = pair(fmt, rows, cols, tokens + rows)
    _, wu, vu = pair(fmt, rows, cols, tokens + rows + 1)
    dh, g, u = (F.bf16_cuda(F.activations(rng, tokens, rows)) for _ in range(3))
    dx, dg, du = qz.gated_ffn_backward(dh, g, u, F.handle(wg), F.handle(wu))
    want = dg.double() @ vg + du.double() @ vu
    terms = dg.double().abs() @ vg.abs() + du.double().abs() @ vu.abs()
    assert bool(((dx.double() - want).abs() <= F.sum_bound(2 * rows, terms) + 2.0 ** -8 * 1.01 * want.abs()).all())


@pytest.mark.parametrize("fmt", list(F.FORMATS))
@pytest.mark.parametrize("shape", PAIRS)
def test_pairs_of_many_tiles(qz, fmt, shape):
    tokens, nout, nsum = shape
    nsum = -(-nsum // F.FORMATS[fmt]) * F.FORMATS[fmt]
    linear_exactly(qz, fmt, tokens, nout + 8, nsum)
    backward_exactly(qz, fmt, tokens, -(-nout // 128) * 128, nsum + 8)


@pytest.mark.parametrize("fmt", list(F.FORMATS))
@pytest.mark.parametrize("shape", [(33, 40008, 128), (250, 20008, 128), (700, 10024, 128)])
def test_gated_pairs_of_many_tiles(qz, fmt, shape):
    gated_exactly(qz, fmt, *shape)
    both_backward(qz, fmt, shape[0], -(-shape[1] // 128) * 128, 200)


@pytest.mark.parametrize("fmt,case", [(f, c) for f in ("mxfp4", "nvfp4") for c in TWO_E2M1] + [("int4", c) for c in TWO_INT4])
def test_two_launches(qz, fmt, case):
    mode, tokens, nout, nsum = case
    if mode == "linear":
        linear_exactly(qz, fmt, tokens, nout, nsum)
    elif mode == "gated":
        gated_exactly(qz, fmt, tokens, nout, nsum)
    else:
        (backward_exactly if mode == "backward" else both_backward)(qz, fmt, tokens, -(-nout // 128) * 128, nsum)


@pytest.mark.parametrize("fmt,group", [("mxfp4", 32), ("nvfp4", 16), ("int4", 32), ("int4", 64), ("int4", 128)])
@pytest.mark.parametrize("shape", FEW)
def test_few_tokens_many_outputs(qz, fmt, group, shape):
    tokens, rows, cols = shape
    cols = -(-cols // group) * group
    linear_exactly(qz, fmt, tokens, rows, cols, group)
    if fmt == "int4":
        linear_exactly(qz, fmt, tokens + 16, rows, cols, group)
    gated_exactly(qz, fmt, tokens, rows, -(-cols // 128) * 128)


@pytest.mark.parametrize("tokens", [1, 8, 17, 40, 300])
@pytest.mark.parametrize("ends", [(-127, -126, -125, -100), (100, 120, 124, 125)])
def test_e8m0_scales_at_both_ends(qz, ends, tokens):
    """2^-127 (weights below bf16's normal range) and 2^125 (6 * 2^125 is the largest in fp32) by every kernel,
    forward and backward."""
    import torch
    rng = np.random.default_rng(tokens)
    w = F.make_weight(rng, "mxfp4", 96, 256)
    k = np.array(ends)[rng.integers(0, 4, (96, 8))]
    w["scales"] = (k + 127).astype(np.uint8)
    w["values"] = w["elements"] * np.repeat(np.ldexp(1.0, k), 32, axis=1)
    scale = 2.0 ** 100 if ends[0] < 0 else 2.0 ** -60
    x, dy = (F.activations(rng, tokens, n) * scale for n in (256, 96))
    h, a = F.handle(w), np.abs(w["values"])
    # (the weights are held exactly: no 2^-17)
    bound = lambda n, terms: F.sum_bound(n, terms) - 2.0 ** -17 * terms  # noqa: E731
    F.assert_within(F.host(qz.linear(F.bf16_cuda(x), h, out_dtype=torch.float32)), x @ w["values"].T, bound(256, np.abs(x) @ a.T))
    F.assert_within(F.host(qz.linear_backward(F.bf16_cuda(dy), h, out_dtype=torch.float32)), dy @ w["values"], bound(96, np.abs(dy) @ a))


@pytest.mark.parametrize("shape", [(1, 70, 512), (7, 300, 640), (16, 96, 2048), (40, 200, 512), (300, 264, 1152)])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_e2m1_weights_are_held_exactly(qz, fmt, shape):
    """Random values against the bound of an fp32 sum alone."""
    import torch
    tokens, rows, cols = shape
    rng = np.random.default_rng(rows)
    w = F.make_weight(rng, fmt, rows, cols)
    x, dy = F.activations(rng, tokens, cols), F.activations(rng, tokens, rows)
    h, a = F.handle(w), np.abs(w["values"])
    for got, want, n, terms in ((qz.linear(F.bf16_cuda(x), h, out_dtype=torch.float32), x @ w["values"].T, cols, np.abs(x) @ a.T),
                                (qz.linear_backward(F.bf16_cuda(dy), h, out_dtype=torch.float32), dy @ w["values"], rows, np.abs(dy) @ a)):
        F.assert_within(F.host(got), want, F.sum_bound(n, terms) - 2.0 ** -17 * terms)


# Calls large enough for the streaming kernel by its estimate: every n-tile count, rows of whole steps of 256
# columns and not, one weight and two, INT4 in two halves.  (mode, format, group, tokens, outputs, columns)
STREAMED = [("linear", "nvfp4", 16, 8, 8192, 4096), ("linear", "mxfp4", 32, 8, 8200, 4064), ("linear", "nvfp4", 16, 9, 32768, 4096),
            ("linear", "mxfp4", 32, 16, 40000, 4064), ("linear", "nvfp4", 16, 16, 40003, 4096), ("gated", "mxfp4", 32, 7, 8192, 4096),
            ("gated", "nvfp4", 16, 8, 8192, 4064), ("gated", "mxfp4", 32, 12, 16384, 4096), ("gated", "nvfp4", 16, 13, 16400, 3872),
            ("linear", "int4", 32, 8, 8192, 1056), ("linear", "int4", 128, 8, 8192, 4096), ("linear", "int4", 32, 16, 8192, 4096),
            ("linear", "int4", 64, 24, 32770, 2048), ("linear", "int4", 128, 31, 32768, 1920), ("linear", "int4", 32, 32, 32768, 2016),
            ("gated", "int4", 128, 9, 8192, 2048), ("gated", "int4", 64, 20, 16384, 1984), ("gated", "int4", 32, 32, 20000, 2048),
            ("linear", "int4", 128, 16, 16384, 8192), ("gated", "int4", 64, 13, 9000, 9088)]


def large(qz, gen, fmt, group, rows, cols):
    """A weight of any codes with scales that are powers of two near 1: the handle's Quantized and the values."""
    import torch
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda", generator=gen)
    k = torch.randint(-2, 2, (rows, cols // group), device="cuda", generator=gen)
    one = torch.ones(1, device="cuda")
    scales = torch.ldexp(one, k) if fmt == "int4" else (k + 127 if fmt == "mxfp4" else (k + 7) << 3).to(torch.uint8)
    q = qz.Quantized(codes, scales, one, qz.FORMATS[fmt], qz.QZ_GRAN_BLOCK, qz.QZ_SCALE_UP, rows, cols, group)
    table = torch.tensor([c - 16 * (c > 7) for c in range(16)] if fmt == "int4" else [*F.E2M1, *-F.E2M1], dtype=torch.float64, device="cuda")
    values = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).reshape(rows, cols // group, group)
    return q, (values * torch.ldexp(one, k).double()[..., None]).reshape(rows, cols)


@pytest.mark.parametrize("case", STREAMED)
def test_streamed(qz, case):
    """Exact sums of ordinary activations, of a token that f16 does not hold (its large value meets codes of 0),
    and beside an output whose scales are 2^100."""
    import torch
    mode, fmt, group, tokens, rows, cols = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens + cols)
    ws = [large(qz, gen, fmt, group, rows, cols) for _ in range(2 if mode == "gated" else 1)]
    for q, v in ws:
        q.codes[:, 0] &= 0xF0
        v[:, 0] = 0
    x = torch.randint(-4, 5, (tokens, cols), device="cuda", generator=gen).double()
    x[:, 0] = 4

    def check(skip=None):
        outs = qz.linear(x.bfloat16(), qz.Weight(ws[0][0]), out_dtype=torch.float32), None
        if mode == "gated":
            outs = qz.gated_ffn(x.bfloat16(), *(qz.Weight(q) for q, _ in ws), save=True)[1:]
        for got, (_, v) in zip(outs, ws):
            want = x @ v.T
            if mode == "gated":
                want = want.float().bfloat16().double()
            same = got.double() == want
            if skip is not None:
                same[:, skip] = True
            assert bool(same.all())

    check()
    x[tokens // 2, 0] = 2.0 ** 45
    check()
    x[tokens // 2, 0] = 4
    if fmt != "nvfp4":  # one output of a tile, most of the way through its sum
        at = (cols // group) * 3 // 4
        ws[0][0].scales[rows - 3, at] = 2.0 ** 100 if fmt == "int4" else 227
        check(skip=rows - 3)
