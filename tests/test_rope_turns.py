"""The rotation table against exact arithmetic: every frequency up to the largest that is taken, as a fraction of a turn
in units of 2^-64.  An angle is position * turn, so half a unit is 2^-34 turns at a position of 2^31."""

from fractions import Fraction

import pytest

import block_quantized_matmul_lwq_b200 as lwq
from block_quantized_matmul_lwq_b200 import build as lwq_build

# pi to 100 digits
TWO_PI = 2 * Fraction(
    int("3141592653589793238462643383279502884197169399375105820974944592307816406286208998628034825342117067"), 10 ** 99)


@pytest.fixture(scope="module", autouse=True)
def built():
    lwq_build.build()


def off(turn, f):
    """Distance of turn from f / (2 pi) modulo 1, in units of 2^-64."""
    d = (turn - Fraction(f) / TWO_PI * 2 ** 64) % 2 ** 64
    return float(min(d, 2 ** 64 - d))


FREQS = [1000003.7, 1048576.0, 1048575.9999999999, 123456.789, 65537.1, 6.283185307179586, 6.283185307179587, 7.5, 1.0,
         0.86, 0.1, 1e-5, 3.3e-12, 1e-19, 5e-324, 0.0, 2.0 ** -61, 2.0 ** 20 - 2.0 ** -33]


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_given_frequencies(sign):
    for i in range(0, len(FREQS), 8):
        part = [sign * f for f in (FREQS[i:i + 8] + [1.0] * 8)[:8]]
        rope = lwq.lwq_rope_init(16, inv_freq=part)
        for f, turn in zip(part, rope.turn):
            assert off(turn, f) <= 0.5 + 2.0 ** -30, f


@pytest.mark.parametrize("rot,base", [(64, 10000.0), (128, 1e6), (128, 1.0), (16, 5e5), (64, 0.01)])
def test_frequencies_of_a_base(rot, base):
    """base^(-2 i / rot) in a floating-point type of 64 bits, off by 2^-62 of its value, so by 2^2 f / (2 pi) units."""
    import math
    rope = lwq.lwq_rope_init(rot, base=base)
    for i in range(rot // 2):
        # the power by its defining equation, f^(rot / 2) = base^-i, to 2^-80
        f = Fraction(math.exp(-2 * i / rot * math.log(base)))
        want = 1 / Fraction(base) ** i
        for _ in range(2):   # Newton
            p = f ** (rot // 2)
            f = f * (1 + (want / p - 1) / (rot // 2))
            f = Fraction(round(f * 2 ** 160), 2 ** 160)
        assert off(rope.turn[i], f) <= 0.5 + float(f) / 6.28 * 2.0 ** 2


def test_frequencies_past_what_a_base_can_hold():
    """Above 256 a frequency of 64 bits is off by 2^-23 of a radian at far positions: such are given themselves."""
    with pytest.raises(lwq.LwqError) as e:
        lwq.lwq_rope_init(128, base=1e-3)
    assert e.value.status == lwq.LWQ_ERR_INVALID_ARG
    lwq.lwq_rope_init(16, inv_freq=[1000.5] * 8)
