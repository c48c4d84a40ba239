"""rope_frequencies against whole-number arithmetic: a frequency's fraction of a turn
to 64 bits, and with it angles to 2^-31 turns at every position.  On the host."""
import random
from fractions import Fraction

import numpy as np
import pytest

from sparse_attention_indexer_idx_gb300 import binding as B

BITS = 400


def arctan_inverse(n):
    """arctan(1 / n) times 2^BITS, off by less than BITS in the last place."""
    x = total = (1 << BITS) // n
    k = 1
    while x:
        x //= n * n
        k += 2
        total += -(x // k) if k % 4 == 3 else x // k
    return total


TWO_PI = Fraction(8 * (4 * arctan_inverse(5) - arctan_inverse(239)), 1 << BITS)      # Machin's formula


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_attention_indexer_idx_gb300 import build
    build.build()


def words(f):
    return [int(x) for x in B.rope_frequencies(2 * len(f), inv_freq=f, device="cpu").numpy().view(np.uint64)]


def apart(a, b):
    """Turns between two angles."""
    d = (a - b) % 1
    return min(d, 1 - d)


rng = random.Random(3)
FREQS = {
    "base 1e4": [10000.0 ** (-i / 64) for i in range(64)],
    "base 5e5": [500000.0 ** (-i / 64) for i in range(64)],
    "base 1e6": [1e6 ** (-i / 32) for i in range(32)],
    "random": [rng.uniform(-8, 8) for _ in range(500)],
    "far": [s * 2.0 ** rng.uniform(-70, 40) for s in (1, -1) for _ in range(200)],
    "ends": [0.0, -0.0, 5e-324, -5e-324, 2.0 ** -64, -2.0 ** -64, 6.283185307179586, -6.283185307179586, 3.0, 1e-300],
}


def test_two_pi():
    assert abs(float(TWO_PI) - 6.283185307179586) < 1e-15


@pytest.mark.parametrize("kind", FREQS)
def test_fractions_of_a_turn_to_64_bits(kind):
    """Half a step of the last bit from rounding to it; 2^-74 and less from a product
    of 106 bits, for up to 2^32 radians a position."""
    for f, w in zip(FREQS[kind], words(FREQS[kind])):
        bound = Fraction(1, 2 ** 65) + abs(Fraction(f)) / 2 ** 104
        assert apart(Fraction(w, 2 ** 64), Fraction(f) / TWO_PI) <= bound, f


@pytest.mark.parametrize("kind", ["base 1e4", "base 5e5", "base 1e6", "random"])
def test_angles_of_far_positions(kind):
    """As the kernel has them: position times word modulo 2^64, its upper 32 bits."""
    for f, w in zip(FREQS[kind], words(FREQS[kind])):
        for pos in (1, 2 ** 22 + 1, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 1999999973):
            angle = Fraction((pos * w % 2 ** 64) >> 32, 2 ** 32)
            assert apart(angle, pos * Fraction(f) / TWO_PI) <= Fraction(1, 2 ** 31), (f, pos)


def test_what_is_refused():
    for bad in (float("nan"), float("inf"), -float("inf")):
        with pytest.raises(B.IdxError):
            words([1.0, bad])
