"""The interpolation by parts against its published formula, pair by pair, also where the slowest pair turns more than
`slow` times over the original positions."""
import math

import pytest


def parts(pairs, base, factor, original, fast=32.0, slow=1.0):
    """Peng et al., YaRN: the ramp between the indices that turn `fast` and `slow` times, held to [0, head dimension - 1]."""
    dim = 2 * pairs

    def correction(turns):
        return dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

    low, high = max(math.floor(correction(fast)), 0), min(math.ceil(correction(slow)), dim - 1)
    if low == high:
        high += 0.001
    out = []
    for i in range(pairs):
        angle = base ** (-2 * i / dim)
        ramp = min(max((i - low) / (high - low), 0.0), 1.0)
        out.append(angle / factor * ramp + angle * (1 - ramp))
    return out


@pytest.mark.parametrize("pairs,base,original", [(32, 10000.0, 4096), (64, 10000.0, 4096), (64, 10000.0, 65536), (64, 10000.0, 131072),
                                                 (16, 10000.0, 65536), (64, 500000.0, 8192), (8, 10000.0, 1 << 20), (1, 10000.0, 4096),
                                                 (64, 1e6, 32768), (32, 10000.0, 128)])
@pytest.mark.parametrize("factor", [1.0, 4.0, 32.0])
def test_parts_is_the_published_formula(pairs, base, original, factor):
    import precision_quantization_gb300 as qz
    got = qz.rotary_turns(pairs, base=base, scaling="parts", factor=factor, original=original).tolist()
    want = parts(pairs, base, factor, original)
    assert len(got) == pairs and all(abs(a - b) <= 1e-12 * b for a, b in zip(got, want)), (got, want)


def test_pairs_that_turn_more_than_slow_are_not_divided_by_all_of_the_factor():
    import precision_quantization_gb300 as qz
    pairs, original, factor = 64, 131072, 4.0
    plain = qz.rotary_turns(pairs).tolist()
    got = qz.rotary_turns(pairs, scaling="parts", factor=factor, original=original).tolist()
    for p, t in zip(plain, got):
        turns = original * p / (2 * math.pi)
        assert turns > 1 and t > 1.3 * p / factor       # every pair turns more than twice: none is divided by all of 4
        if turns > 32 * 10000.0 ** (1 / pairs):
            assert abs(t - p) <= 1e-12 * p


def test_parts_refuses_bases_that_order_the_pairs_the_other_way():
    import precision_quantization_gb300 as qz
    for base in (1.0, 0.5, 1e-4):
        with pytest.raises(ValueError):
            qz.rotary_turns(8, base=base, scaling="parts", factor=2.0, original=4096)
    assert qz.rotary_turns(8, base=0.5).numel() == 8
