"""The example that runs norm, projections, append and attention together."""
import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,cache,heads,kv_heads,dim", [("nvfp4", "e4m3", 16, 4, 64), ("mxfp4", "int8", 8, 8, 128), ("int4", "e5m2", 6, 1, 96)])
def test_attention_block(fmt, cache, heads, kv_heads, dim):
    import __graft_entry__
    __graft_entry__.build_library()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import attention_block as ex
    # Each stage is compared on its own inputs: a bf16 rounding of its result (2^-8 at most), for the attention also one
    # of its weights to 11 bits (2^-11), for y one of the product and one of the sum.
    for name, e in ex.run(fmt, cache, heads, kv_heads, dim).items():
        assert e <= 2.0 ** -8 + 2.0 ** -10 if name.startswith("attention") else e <= 2 * 2.0 ** -8, (name, e)
