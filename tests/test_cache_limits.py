"""The largest and smallest arguments of the attention to the 8-bit cache, without a GPU."""
import math

from test_cache_args import FAKE, batch, cache, qz  # noqa: F401


def test_scales_that_overflow_in_base_two_are_refused(qz):  # noqa: F811
    """The scores are kept in units of log 2: a scale times 1 / log 2 has to be a number too.  (No sequences: nothing is launched.)"""
    call = lambda s: qz.qz_cache_attention(cache(qz), batch(qz, n=0), FAKE, 256, 64, 0, 4, s, 0, FAKE, 256, 64, None, 0, None, 0)  # noqa: E731
    for s in (2.0 ** 127 * (1 + 2.0 ** -23), 3.4e38, math.inf, math.nan, 0.0, -1.0):
        assert call(s) == qz.QZ_ERR_SHAPE, s
    for s in (2.0 ** 127, 1.0, 2.0 ** -149):
        assert call(s) == qz.QZ_OK, s
