"""blkattn_rope_phases rounds to the nearest phase over its whole range.  No
GPU.  The exact value is taken with rationals; pi to 80 digits is off by less
than 2^-260, the table's own constant by 2^-128 relative, at most 2^-62 units."""
import random
from fractions import Fraction

import pytest

from exact_blocked_attention_gb300 import blkattn
from exact_blocked_attention_gb300 import build as libbuild

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    blkattn.load()


@pytest.mark.parametrize("lo,hi", [(4.0, 8.0), (1.0, 4.0), (0.5, 1.0), (1e-3, 0.5), (1e-12, 1e-6)])
def test_phases_are_rounded_to_the_nearest(lo, hi):
    rng = random.Random(int(hi * 1000))
    angles = [rng.uniform(lo, hi) * rng.choice((1, -1)) for _ in range(400)] + [lo, hi, -lo, -hi]
    for a, f in zip(angles, blkattn.rope_phases(angles, device="cpu").tolist()):
        d = (f - Fraction(a) * 2 ** 64 / TWO_PI) % 2 ** 64
        assert min(d, 2 ** 64 - d) <= Fraction(1, 2) + Fraction(1, 2 ** 60), a
