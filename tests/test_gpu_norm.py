"""Layer norm and its gradients on the GPU, against 64-bit references."""
import numpy as np
import pytest

import ffn_util as F

pytestmark = pytest.mark.gpu

# one row and one column, odd widths, each number of threads a row takes, a row read from memory
# again (> 16384), more rows than one pass of the grid
SHAPES = [(1, 1), (3, 2), (7, 31), (5, 512), (300, 520), (64, 1000), (33, 2048), (9, 4095), (700, 4096),
          (20, 8200), (6, 16384), (4, 16385), (3, 20000), (5000, 64)]


@pytest.fixture(scope="module")
def qz():
    import __graft_entry__
    __graft_entry__.build_library()
    import precision_quantization_gb300 as qz
    qz.lib()
    return qz


def tensor(a, dtype, pad=0):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    if pad:
        big = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), dtype=t.dtype)
        big[:, :a.shape[1]] = t
        return big.cuda()[:, :a.shape[1]]
    return t.cuda()


def inputs(rng, rows, cols, dtype):
    x = rng.normal(1.0, 2.0, (rows, cols))
    dy = rng.normal(0, 1, (rows, cols))
    x, dy = (F.bf16_round(v) if dtype == "bf16" else v.astype(np.float32).astype(np.float64) for v in (x, dy))
    w, b = (v.astype(np.float32).astype(np.float64) for v in (rng.normal(1, 0.3, cols), rng.normal(0, 0.3, cols)))
    return x, dy, w, b


def forward(x, w, b, eps):
    mean = x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    return (x - mean) * rstd * w + b, mean, rstd


def f32(v):
    import torch
    return torch.from_numpy(v.astype(np.float32)).cuda()


# A row sum runs as at most 16 adds in a thread (cols / 1024 for rows read again), 10 more over
# the threads, so its relative error is under (16 + 10 + cols / 1024) 2^-24 of the sum of
# magnitudes; U bounds what that does to mean, rstd and n, with a factor of two to spare.
def u_of(cols):
    return 2 * (32 + cols / 1024) * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(qz, dtype, affine, shape):
    rows, cols = shape
    rng = np.random.default_rng(rows + cols)
    x, _, w, b = inputs(rng, rows, cols, dtype)
    y, mean, rstd = qz.layer_norm(tensor(x, dtype), f32(w) if affine else None, f32(b) if affine else None)
    if not affine:
        w, b = np.ones(cols), np.zeros(cols)
    want, m, r = forward(x, w, b, 1e-5)
    u = u_of(cols)
    big = np.abs(x).max(-1, keepdims=True)
    assert np.abs(F.host(mean) - m[:, 0]).max() <= u * big.max()
    # the mean's error enters the squares' sum twice and rstd falls as its root
    rel = u * (1 + big * r)
    F.assert_within(F.host(rstd), r[:, 0], (rel * r)[:, 0])
    bound = rel * (np.abs(want - b) + np.abs(w) * (1 + big * r)) + 2.0 ** -22 * (np.abs(want) + np.abs(b))
    F.assert_within(F.host(y), want, bound + (F.bf16_bound(want) if dtype == "bf16" else 0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(qz, dtype, affine, shape):
    rows, cols = shape
    rng = np.random.default_rng(rows * 7 + cols)
    x, dy, w, _ = inputs(rng, rows, cols, dtype)
    if not affine:
        w = np.ones(cols)
    _, m, r = forward(x, w, 0, 1e-5)
    m, r = (v.astype(np.float32).astype(np.float64) for v in (m, r))
    args = (tensor(dy, dtype), tensor(x, dtype), f32(m[:, 0]), f32(r[:, 0]), f32(w) if affine else None)
    dx, dw, db = qz.layer_norm_backward(*args)
    n = (x - m) * r
    t = dy * w
    want = r * (t - t.mean(-1, keepdims=True) - n * (t * n).mean(-1, keepdims=True))
    u = u_of(cols)
    mag = np.abs(t) + np.abs(t).mean(-1, keepdims=True) + np.abs(n) * np.abs(t * n).mean(-1, keepdims=True)
    bound = (u + 2.0 ** -20) * r * mag * (1 + np.abs(m) * r)
    F.assert_within(F.host(dx), want, bound + (F.bf16_bound(want) if dtype == "bf16" else 0), "dx")
    # column sums: at most rows adds in a chain, n with three roundings
    cu = (rows + 64) * 2.0 ** -24
    scale = (np.abs(dy) * (np.abs(n) + np.abs(m) * r)).sum(0)
    F.assert_within(F.host(dw), (dy * n).sum(0), cu * scale + 1e-30, "dweight")
    F.assert_within(F.host(db), dy.sum(0), cu * np.abs(dy).sum(0) + 1e-30, "dbias")
    dx2, none, _ = qz.layer_norm_backward(*args, params=False)
    assert none is None and np.array_equal(F.host(dx2), F.host(dx))
    again = qz.layer_norm_backward(*args)
    assert all(np.array_equal(F.host(p), F.host(q)) for p, q in zip(again, (dx, dw, db)))


def placed(a, dtype, lead, ld, fill):
    """The matrix as a view: `lead` values into a buffer of `fill`, rows `ld` apart."""
    import torch
    rows, cols = a.shape
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    buf = torch.full((lead + rows * ld + 8,), fill, dtype=dt, device="cuda")
    view = buf.as_strided((rows, cols), (ld, 1), lead)
    view.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda())
    return buf, view


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lead,pad", [(0, 0), (1, 0), (3, 2), (6, 5), (7, 8)])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (2, 15), (17, 63), (1300, 37), (310, 505), (300, 1021), (160, 2047), (170, 4095),
                                   (30, 8185), (18, 16377), (9, 16383)])
def test_backward_rows_at_any_place(qz, dtype, lead, pad, shape):
    """Rows that start anywhere between two 16-byte boundaries: the values around them (NaN) stay
    out of the results and what surrounds dx stays as it was."""
    rows, cols = shape
    rng = np.random.default_rng(rows + 3 * cols + lead)
    x, dy, w, _ = inputs(rng, rows, cols, dtype)
    _, m, r = forward(x, w, 0, 1e-5)
    m, r = (v.astype(np.float32).astype(np.float64) for v in (m, r))
    _, vx = placed(x, dtype, lead, cols + pad, float("nan"))
    _, vdy = placed(dy, dtype, lead + 8, cols + pad + 8, float("nan"))
    buf, vdx = placed(np.zeros_like(x), dtype, lead, cols + pad, 5.0)
    dw, db = f32(np.zeros(cols)), f32(np.zeros(cols))
    qz.layer_norm_backward(vdy, vx, f32(m[:, 0]), f32(r[:, 0]), f32(w), out=(vdx, dw, db))
    n = (x - m) * r
    t = dy * w
    want = r * (t - t.mean(-1, keepdims=True) - n * (t * n).mean(-1, keepdims=True))
    mag = np.abs(t) + np.abs(t).mean(-1, keepdims=True) + np.abs(n) * np.abs(t * n).mean(-1, keepdims=True)
    bound = (u_of(cols) + 2.0 ** -20) * r * mag * (1 + np.abs(m) * r)
    F.assert_within(F.host(vdx), want, bound + (F.bf16_bound(want) if dtype == "bf16" else 0), "dx")
    cu = (rows + 64) * 2.0 ** -24
    F.assert_within(F.host(dw), (dy * n).sum(0), cu * (np.abs(dy) * (np.abs(n) + np.abs(m) * r)).sum(0) + 1e-30, "dweight")
    F.assert_within(F.host(db), dy.sum(0), cu * np.abs(dy).sum(0) + 1e-30, "dbias")
    vdx.fill_(5.0)
    assert bool((buf == 5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(900, 2056), (901, 3071), (640, 4104), (641, 6143), (800, 8200), (330, 10239), (320, 12288), (310, 12296)])
def test_threads_between_powers_of_two(qz, dtype, shape):
    test_forward(qz, dtype, True, shape)
    test_backward(qz, dtype, True, shape)


def test_gradient_is_the_difference(qz):
    """sum(dy * y) moved by +-h along a direction, through the fp32 kernel itself."""
    rng = np.random.default_rng(4)
    x, dy, w, b = inputs(rng, 6, 300, "f32")
    d, h = rng.normal(size=x.shape), 1e-2
    dw_dir, db_dir = rng.normal(size=300), rng.normal(size=300)

    def f(s):
        y = qz.layer_norm(tensor(x + s * h * d, "f32"), f32(w + s * h * dw_dir), f32(b + s * h * db_dir))[0]
        return (dy * F.host(y)).sum()

    _, mean, rstd = qz.layer_norm(tensor(x, "f32"), f32(w), f32(b))
    dx, dw, db = qz.layer_norm_backward(tensor(dy, "f32"), tensor(x, "f32"), mean, rstd, f32(w))
    slope = (F.host(dx) * d).sum() + (F.host(dw) * dw_dir).sum() + (F.host(db) * db_dir).sum()
    # y errs by 2^-20 of its size at most, so each f by 2^-20 sum |dy y| (about 2000 * 2^-20), the
    # quotient by that over h; the third derivative adds h^2 times the same size
    size = np.abs(dy).sum() * 4
    assert abs((f(1) - f(-1)) / (2 * h) - slope) <= size * (2.0 ** -20 / h + 2 * h * h)


@pytest.mark.parametrize("pad", [3, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides(qz, dtype, pad):
    import torch
    rng = np.random.default_rng(pad)
    x, dy, w, b = inputs(rng, 40, 640, dtype)
    y, mean, rstd = qz.layer_norm(tensor(x, dtype, pad), f32(w), f32(b))
    y2, _, _ = qz.layer_norm(tensor(x, dtype), f32(w), f32(b))
    F.assert_within(F.host(y), F.host(y2), 2.0 ** -18 * (1 + np.abs(F.host(y2))) + (2 * F.bf16_bound(F.host(y2)) if dtype == "bf16" else 0))
    big = torch.full((40, 640 + pad), 5.0, dtype=y.dtype, device="cuda")
    dw, db = torch.empty(640, device="cuda"), torch.empty(640, device="cuda")
    qz.layer_norm_backward(tensor(dy, dtype, pad), tensor(x, dtype), mean, rstd, f32(w), out=(big[:, :640], dw, db))
    dx, dw2, db2 = qz.layer_norm_backward(tensor(dy, dtype), tensor(x, dtype), mean, rstd, f32(w))
    F.assert_within(F.host(big[:, :640]), F.host(dx), 2.0 ** -16 * (1 + np.abs(F.host(dx))) + (2 * F.bf16_bound(F.host(dx)) if dtype == "bf16" else 0))
    assert bool((big[:, 640:] == 5).all())
    F.assert_within(F.host(dw), F.host(dw2), 2.0 ** -16 * (1 + np.abs(F.host(dw2))))


def test_rows_and_specials(qz):
    """No rows; a constant row (zero variance); a NaN and an Inf stay in their rows."""
    import torch
    e = torch.empty((0, 128), device="cuda")
    y, mean, rstd = qz.layer_norm(e)
    assert y.shape == (0, 128) and mean.shape == (0,)
    dx, dw, db = qz.layer_norm_backward(e, e, mean, rstd)
    assert dx.shape == (0, 128) and bool((dw == 0).all()) and bool((db == 0).all())
    x = torch.randn(4, 256, device="cuda")
    x[1] = 3.0
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    y, mean, rstd = qz.layer_norm(x)
    assert bool(torch.isfinite(y[0]).all()) and bool((y[1] == 0).all())
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).all())
    assert abs(float(rstd[1]) - 1e-5 ** -0.5) < 1e-3
