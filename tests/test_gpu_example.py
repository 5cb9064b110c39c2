"""The example that runs norm, gated block, projection and their gradients together."""
import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "int4"])
@pytest.mark.parametrize("tokens", [5, 300])
def test_feed_forward_block(fmt, tokens):
    import __graft_entry__
    __graft_entry__.build_library()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import feed_forward_block as ex
    # Five tensors in a row are rounded to bf16 (the norm's output, h, the projection, dn, dx), each by
    # 2^-9 of its size at rms; a value passes through at most all of them: 5 * 2^-9 bounds the
    # relative 2-norm of any of the results.
    for name, e in ex.run(fmt, tokens=tokens).items():
        assert e <= 5 * 2.0 ** -9, (name, e)
