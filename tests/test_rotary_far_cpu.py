"""Frequencies stretched by factors whose powers leave 64 bits (no GPU)."""
from fractions import Fraction
import math

import pytest

paro = pytest.importorskip("rotation_int4_weight_amd")
pytest.importorskip("torch")


@pytest.mark.parametrize("rot,base,factor", [(4, 1e4, 1e200), (4, 1e300, 1e200), (6, 1e308, 1e300), (128, 1e308, 4.0),
                                             (512, 1e4, 8.0), (4, 1e4, 1.0)])
def test_a_scaled_base_past_the_range(rot, base, factor):
    """The fastest pair stays and the slowest is divided by factor, also where base * factor^(rot / (rot - 2)) is no
    64-bit number.  In logarithms, whose 2^-53 of at most 1420 are 1.6e-13 of the frequency; a frequency under half of
    the least 64-bit number, 2^-1075, rounds to 0 (1e-150 / 1e200, 1e-205 / 1e300)."""
    f, magnitude = paro.paro_rotary_frequencies(rot, base=base, kind="base", factor=factor, device="cpu")
    assert f[0] == 1.0 and magnitude == 1.0
    for i, x in enumerate(f.tolist()):
        log = -float(Fraction(2 * i, rot)) * math.log(base) - float(Fraction(2 * i, rot - 2)) * math.log(factor)
        if log < -1075 * math.log(2):
            assert x == 0.0
            continue
        assert x > 0 and abs(math.log(x) - log) <= 1e-12, (i, x)
