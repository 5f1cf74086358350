"""The fixed-point fraction of a turn that gqa_qk_norm_rope gives a frequency,
restated in float64 and exact fractions (no GPU)."""
from fractions import Fraction

import numpy as np

from test_gpu_norm_rope_angles import FREQS, TWO_PI


def test_the_fraction_itself():
    """The two-part product, restated in float64: within 2^-63.9 turns for
    every frequency up to 2^40, where the rounded product is not."""
    hi = 0.15915494309189535
    lo = float(1 / TWO_PI - Fraction(hi))
    rng = np.random.default_rng(0)
    freqs = [float(np.float32(f)) for f in FREQS] + \
        [float(np.float32(s * 2.0 ** e)) for s, e in zip(rng.choice([-1, 1], 400), rng.uniform(-60, 40, 400))]
    worst = worst_rounded = Fraction(0)
    for f in freqs:
        t = f * hi
        e = float(Fraction(f) * Fraction(hi) - Fraction(t))           # exact (an fma)
        r = t - round(t)                                              # exact
        rest = float(Fraction(f) * Fraction(lo) + Fraction(e))        # one rounding (an fma)
        got = Fraction(round(Fraction(r) * 2 ** 64) + round(Fraction(rest) * 2 ** 64), 2 ** 64)
        exact = Fraction(f) / TWO_PI
        off = got - exact
        worst = max(worst, abs(off - round(off)))
        off = Fraction(t) - exact
        worst_rounded = max(worst_rounded, abs(off - round(off)))
    assert worst <= Fraction(2.0 ** -63.9)
    assert worst_rounded > Fraction(2) ** -30
