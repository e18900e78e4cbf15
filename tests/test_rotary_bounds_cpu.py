"""What an angle from 64-bit fractions of a turn is off by, in whole fractions."""
import math
import random
from fractions import Fraction

from verify_dspark_markov_step_gb300 import rotary

TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889")


def angle(position, radians):
    """position * radians modulo a turn, in radians (within half a turn)."""
    t = position * radians / TWO_PI % 1
    return float((t - 1 if t > Fraction(1, 2) else t) * TWO_PI)


def test_the_angle_is_off_by_the_turns_own_rounding():
    """position * 2^-65 turns, and no more; so far out that no position of a model comes
    near, that is much of a turn."""
    rng = random.Random(1)
    largest = 0.0
    for w in [1.0, 0.1, 3e-6] + rotary.frequencies(128, 5e5)[0]:
        turns = rotary.turns_of([w])[0]
        exact = Fraction(w) / TWO_PI
        for bits in (1, 20, 31, 40, 53, 62):
            p = rng.randrange(2 ** (bits - 1), 2 ** bits)
            off = (Fraction(p * turns % 2 ** 64, 2 ** 64) - p * exact) % 1
            off = min(off, 1 - off)
            assert off <= Fraction(p, 2 ** 65)
            if bits == 62:
                largest = max(largest, float(off))
    assert 2.0 ** -5 < largest <= 2.0 ** -3


def test_a_frequency_in_64_bits_is_off_too():
    """The frequencies are doubles: a relative 2^-50 of the power at most, which at one radian
    a position and 2^40 positions is 2^-10 of a radian."""
    for i, w in enumerate(rotary.frequencies(128, 1e4)[0]):
        # 10^(-i / 16) in whole numbers: w^16 is 10^-i
        r = Fraction(w) ** 16 * 10 ** i
        assert abs(math.log(float(r))) <= 16 * 2.0 ** -50 and abs(r - 1) <= 17 * Fraction(1, 2 ** 50)
