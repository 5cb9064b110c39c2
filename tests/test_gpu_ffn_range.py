"""Products with 4-bit weights where magnitudes lie far apart: activations of one token, the scales of
neighbouring rows, scale bytes that the quantizer does not write for finite input."""
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


def bound(w, tokens, k, terms):
    """F.sum_bound for weights that are held exactly; its 2^-17 belongs to INT4 weights on the
    tensor-core tiles alone (up to 4 tokens of up to 4096 columns never take them), as the sum of two
    bf16 values."""
    two_terms = w["fmt"] == "int4" and tokens > 4
    return F.sum_bound(k, terms) - (0 if two_terms else 2.0 ** -17) * terms + 2.0 ** -140


def linear(qz, x, w):
    import torch
    return F.host(qz.linear(F.bf16_cuda(x), F.handle(w), out_dtype=torch.float32))


# one token, one n-tile of eight, two and more, whichever kernel they take at these sizes
TOKENS = [1, 7, 16, 17, 32, 33]


@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("fmt", list(F.FORMATS))
def test_small_activations_beside_a_large_one(qz, fmt, tokens):
    """x = (2^e, 1, ..., 1) and weights (0, 1, ..., 1): the sum is that of the ones, whatever e is."""
    group = F.FORMATS[fmt]
    w = F.make_weight(np.random.default_rng(0), fmt, 40, 256)
    one = 1 if fmt == "int4" else 2  # the code of 1
    nib = np.full((40, 256), one, np.uint8)
    nib[:, ::group] = 0
    w["codes"] = (nib[:, 0::2] | (nib[:, 1::2] << 4)).astype(np.uint8)
    w["scales"] = np.full_like(w["scales"], {"int4": 1.0, "mxfp4": 127, "nvfp4": 0x38}[fmt])
    w["ts"] = np.float32(1)
    for e in (10, 30, 31, 32, 40, 100, 127):
        x = np.ones((tokens, 256))
        x[:, ::group] = 2.0 ** e
        assert np.array_equal(linear(qz, x, w), np.full((tokens, 40), 256.0 - 256 // group)), e


@pytest.mark.parametrize("cols", [512, 1152])
@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("fmt", list(F.FORMATS))
def test_activations_of_any_range(qz, fmt, tokens, cols):
    """Channels up to 2^100 times the others, on codes of 0 in half of the rows."""
    rng = np.random.default_rng(tokens + cols)
    w = F.make_weight(rng, fmt, 70, cols)
    at = rng.integers(0, cols, 9)
    nib = np.stack((w["codes"] & 15, w["codes"] >> 4), -1).reshape(70, cols)
    nib[::2, at] = 0
    w["codes"] = (nib[:, 0::2] | (nib[:, 1::2] << 4)).astype(np.uint8)
    w["values"][::2, at] = 0
    for base, e in ((1.0, 20), (1.0, 29), (2.0 ** -90, 33), (2.0 ** 60, 45), (2.0 ** -60, 100)):
        x = F.activations(rng, tokens, cols, scale=base)
        x[: (tokens + 1) // 2, at] *= 2.0 ** e  # the other tokens have no such channels
        a = np.abs(w["values"])
        F.assert_within(linear(qz, x, w), x @ w["values"].T, bound(w, tokens, cols, np.abs(x) @ a.T), e)


@pytest.mark.parametrize("tokens", [1, 8, 16])
@pytest.mark.parametrize("fmt", ["mxfp4", "int4"])
def test_large_activations_times_the_smallest_scales(qz, fmt, tokens):
    """Scales near 2^-126 on activations near 2^70, beside one of 2^100 on a code of 0."""
    rng = np.random.default_rng(tokens)
    w = F.make_weight(rng, fmt, 33, 256)
    w["codes"][:, 0] &= 0xF0
    w["elements"][:, 0] = 0
    k = rng.integers(-126, -120, w["scales"].shape)
    w["scales"] = np.ldexp(1.0, k).astype(np.float32) if fmt == "int4" else (k + 127).astype(np.uint8)
    w["values"] = w["elements"] * np.repeat(np.ldexp(1.0, k), w["group"], axis=1)
    x = F.activations(rng, tokens, 256, scale=2.0 ** 70)
    x[:, 0] = 2.0 ** 100
    F.assert_within(linear(qz, x, w), x @ w["values"].T, bound(w, tokens, 256, np.abs(x) @ np.abs(w["values"]).T))


@pytest.mark.parametrize("tokens", [1, 9])
@pytest.mark.parametrize("fmt", list(F.FORMATS))
def test_gated_activations_of_any_range(qz, fmt, tokens):
    """The same sums for gate and up: the kept pre-activations."""
    rng = np.random.default_rng(tokens)
    wg, wu = (F.make_weight(rng, fmt, 40, 512) for _ in range(2))
    for w in (wg, wu):
        w["codes"][:, 7] = 0
        w["values"][:, 14:16] = 0
    x = F.activations(rng, tokens, 512)
    x[:, 14] *= 2.0 ** 45
    _, g, u = qz.gated_ffn(F.bf16_cuda(x), F.handle(wg), F.handle(wu), save=True)
    for got, w in ((g, wg), (u, wu)):
        want = x @ w["values"].T
        F.assert_within(F.host(got), want, F.bf16_bound(want) + 1.01 * bound(w, tokens, 512, np.abs(x) @ np.abs(w["values"]).T))


@pytest.mark.parametrize("fmt", list(F.FORMATS))
def test_nonfinite_beside_a_wide_token(qz, fmt):
    """NaN and Inf stay in their tokens where another token spans many binades."""
    rng = np.random.default_rng(5)
    w = F.make_weight(rng, fmt, 50, 256)
    x = F.activations(rng, 6, 256)
    x[1, 3], x[1, 4] = 2.0 ** 50, 2.0 ** -50
    clean = linear(qz, x, w)
    x[0, 9], x[4, 10] = np.nan, np.inf
    got = linear(qz, x, w)
    assert np.isnan(got[0]).all() and not np.isfinite(got[4]).any()
    keep = [1, 2, 3, 5]
    assert np.array_equal(got[keep], clean[keep])


@pytest.mark.parametrize("where", ["rows", "blocks"])
@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("fmt", ["mxfp4", "int4"])
def test_scales_far_apart(qz, fmt, tokens, where):
    """Scales near 2^100 in every fourth output (or on blocks of zeros in every fourth, and on real
    weights in one), 2^-100 in the others: each output has the accuracy of its own products."""
    rng = np.random.default_rng(tokens)
    cols = 1024
    w = F.make_weight(rng, fmt, 83, cols)
    blocks = cols // w["group"]
    k = rng.integers(-104, -96, (83, blocks))
    if where == "rows":
        k[1::4] = rng.integers(96, 104, (len(k[1::4]), blocks))
    else:
        high = rng.integers(0, blocks, 83)
        k[np.arange(83), high] = 110
        for r in range(83):
            if r != 40:
                part = slice(high[r] * w["group"] // 2, (high[r] + 1) * w["group"] // 2)
                w["codes"][r, part] = 0
                w["elements"][r, 2 * part.start:2 * part.stop] = 0
    w["scales"] = np.ldexp(1.0, k).astype(np.float32) if fmt == "int4" else (k + 127).astype(np.uint8)
    w["values"] = w["elements"] * np.repeat(np.ldexp(1.0, k), w["group"], axis=1)
    x = F.activations(rng, tokens, cols)
    F.assert_within(linear(qz, x, w), x @ w["values"].T, bound(w, tokens, cols, np.abs(x) @ np.abs(w["values"]).T))


@pytest.mark.parametrize("cols", [512, 544])  # scales loaded together, or one at a time
@pytest.mark.parametrize("tokens", [1, 17, 40, 300])
@pytest.mark.parametrize("fmt", list(F.FORMATS))
def test_scale_is_nan(qz, fmt, tokens, cols):
    """A NaN scale makes its output NaN (backward: the gradients of its columns) and nothing else."""
    import torch
    group = 32 if fmt == "int4" else F.FORMATS[fmt]
    rng = np.random.default_rng(cols)
    w = F.make_weight(rng, fmt, 70, cols, group)
    x, dy = F.activations(rng, tokens, cols), F.activations(rng, tokens, 70)
    clean = linear(qz, x, w)
    clean_dx = F.host(qz.linear_backward(F.bf16_cuda(dy), F.handle(w), out_dtype=torch.float32))
    w["scales"][5, 3] = w["scales"][64, 0] = {"mxfp4": 255, "nvfp4": 0x7F, "int4": np.nan}[fmt]
    got = linear(qz, x, w)
    assert np.isnan(got[:, [5, 64]]).all()
    rest = np.setdiff1d(np.arange(70), [5, 64])
    F.assert_within(got[:, rest], clean[:, rest], 2 * bound(w, tokens, cols, np.abs(x) @ np.abs(w["values"][rest]).T))
    dx = F.host(qz.linear_backward(F.bf16_cuda(dy), F.handle(w), out_dtype=torch.float32))
    hit = np.zeros(cols, bool)
    hit[:group] = hit[3 * group:4 * group] = True
    assert np.isnan(dx[:, hit]).all() and np.array_equal(dx[:, ~hit], clean_dx[:, ~hit])
    _, g, u = qz.gated_ffn(F.bf16_cuda(x), F.handle(w), F.handle(w), save=True)
    assert np.isnan(F.host(g)[:, [5, 64]]).all() and np.isfinite(F.host(u)[:, rest]).all()


@pytest.mark.parametrize("tokens", [1, 17, 300])
def test_every_e4m3_scale(qz, tokens):
    """All 254 finite E4M3 bytes, the negative ones too, have the value that dequantize gives them."""
    import torch
    rng = np.random.default_rng(tokens)
    w = F.make_weight(rng, "nvfp4", 64, 256)
    b = rng.permutation(np.concatenate([np.arange(0x7F), np.arange(0x80, 0xFF)]).repeat(5)[:1024]).reshape(64, 16)
    w["scales"] = b.astype(np.uint8)
    k = F.e4m3_value(b & 127) * np.where(b > 127, -1, 1) * np.float64(w["ts"])
    w["values"] = w["elements"] * np.repeat(k, 16, axis=1)
    x, dy = F.activations(rng, tokens, 256), F.activations(rng, tokens, 64)
    a = np.abs(w["values"])
    F.assert_within(linear(qz, x, w), x @ w["values"].T, bound(w, tokens, 256, np.abs(x) @ a.T))
    dx = F.host(qz.linear_backward(F.bf16_cuda(dy), F.handle(w), out_dtype=torch.float32))
    F.assert_within(dx, dy @ w["values"], bound(w, tokens, 64, np.abs(dy) @ a))
