"""Products with 4-bit weights and layer norm on a stream that is not the current one."""
import numpy as np
import pytest

import ffn_util as F

pytestmark = pytest.mark.gpu


def test_same_results_on_a_busy_side_stream():
    """The side stream is behind by a millisecond while the current one takes and overwrites memory:
    neither sees the other's blocks."""
    import torch

    import __graft_entry__
    __graft_entry__.build_library()
    import precision_quantization_gb300 as qz
    rng = np.random.default_rng(2)
    gate, up, down = (F.handle(F.make_weight(rng, "nvfp4", *s)) for s in ((1024, 512), (1024, 512), (512, 1024)))
    x, dy = (F.bf16_cuda(F.activations(rng, 700, 512)) for _ in range(2))

    def step(**k):
        n, mean, rstd = qz.layer_norm(x, **k)
        h, g, u = qz.gated_ffn(n, gate, up, save=True, **k)
        y = qz.linear(h, down, **k)
        dh = qz.linear_backward(dy, down, **k)
        dn, dg, du = qz.gated_ffn_backward(dh, g, u, gate, up, **k)
        return (y, h, g, u, dn, dg, du, mean, rstd, *qz.layer_norm_backward(dn, x, mean, rstd, **k))

    want = step()
    sizes = {t.numel() * t.element_size() for t in want} | {qz.qz_layer_norm_backward_workspace(700, 512)}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        at = {t.data_ptr() for t in freed}
        del freed
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000)
        got = step(stream=side)
        for n in sizes:
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN in bf16 and fp32
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert not at & {t.data_ptr() for t in got}
