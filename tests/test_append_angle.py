"""The angle of an append's turn as its kernel forms it, in the same integer and fp32 steps, against exact fractions."""
from fractions import Fraction

import numpy as np
import pytest


def _angle(pos, turn):
    """The fraction of a turn in [-1/2, 1/2): the upper 32 bits of the product, rounded, as fp32."""
    f = ((pos * turn + 0x80000000) >> 32) & 0xFFFFFFFF
    return np.float32(f - 2**32 if f >= 2**31 else f) * np.float32(2.0**-32)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("base", [1.5, 10000.0, 500000.0, 3.0e38])
def test_angle_is_within_the_stated_bound_at_every_position(base, D):
    from kv_cache_decode_flash_gb300 import kvc

    rng = np.random.default_rng(5)
    positions = [0, 1, 2, 3, 2**23 - 1, 2**23 + 1, 2**31 - 1] + [int(2 ** x) for x in rng.uniform(0, 31, 300)]
    worst = Fraction(0)
    for turn in kvc.kvc_debug_rope_turns(base, D):
        for p in positions:
            exact = Fraction(p * turn, 2**64)
            off = abs(Fraction(float(_angle(p, turn))) - exact) % 1
            worst = max(worst, min(off, 1 - off))
    # 2^-33 from the upper 32 bits and half a step of fp32 below 1/2, 2^-26: 1.51e-8, and 2^-64 a position from the turn itself
    assert worst <= Fraction(1, 2**33) + Fraction(1, 2**26)
    assert float(worst) + 2.0**-33 < 1.6e-8
