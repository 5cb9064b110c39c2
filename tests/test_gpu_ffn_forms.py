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
