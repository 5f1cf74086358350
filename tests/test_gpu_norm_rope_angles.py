"""The angles of gqa_qk_norm_rope for frequencies of any size.

The rotation of (1, 0) is (cos a, sin a) of the exact angle.  Bound, in turns:
the frequency's 64-bit fraction is within 2^-63.9, times a position of at most
2^31: 2^-32.9; the product's lower half is dropped: 2^-32; the rest, a signed
half turn below 1, is rounded to fp32: 2^-25 half turns.  Together below 2^-25.9
turns, 2 pi of which are 2^-23.2 radians; a cosine or sine rounds twice more (2
ulp of at most 2^-24 each): below 2^-21.9 in all, held to 2^-21.8."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TWO_PI = Fraction(2) * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
POSITIONS = [0, 1, -1, 2, 4095, -4096, 10 ** 6 + 3, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31]
FREQS = [1.0, 0.999, 3.1415927, 6.2831855, 6.2831850, 12.566371, 7.0, 100.0, 12345.678, 1e6, 3.3e7, 2.0 ** 31 + 256,
         2.0 ** 40, -1.0, -6.2831855, -1e6, -2.0 ** 40, 1e-3, 1e-6, -1e-6, 2.0 ** -40, -2.0 ** -60, 1e-30, -1e-30,
         1e-44, 0.0, 0.5, 1.5707964, -1.5707964, 2.0 ** 20 * 6.2831855, 9.2e11, -7.7e11]


@pytest.mark.parametrize("d,interleaved", [(2 * len(FREQS), False), (2 * len(FREQS), True), (2 * len(FREQS) + 2, False)])
def test_the_fraction_of_a_turn(cuda_lib, d, interleaved):
    """(The last width runs the row kernel.)"""
    fr = torch.tensor(FREQS, dtype=torch.float32)
    half, T = len(FREQS), len(POSITIONS)
    assert half == 32
    u = [2 * i if interleaved else i for i in range(half)]
    v = [2 * i + 1 if interleaved else half + i for i in range(half)]
    x = torch.zeros(1, T, 3, d)
    x[..., u] = 1.0
    pos = torch.tensor([POSITIONS], dtype=torch.int64).to(torch.int32)
    q, k, _ = cuda_lib.qk_norm_rope(x.view(1, T, -1).to(DEV), 1, 1, d, inv_freq=fr.to(DEV), interleaved=interleaved,
                                    positions=pos.to(DEV))
    for y in (q, k):
        got = y[0, 0].double().cpu().numpy()
        for j, pj in enumerate(POSITIONS):
            for i, f in enumerate(fr.tolist()):
                a = Fraction(pj) * Fraction(f)
                a = float(a - TWO_PI * round(a / TWO_PI))
                err = max(abs(got[j, u[i]] - math.cos(a)), abs(got[j, v[i]] - math.sin(a)))
                assert err <= 2.0 ** -21.8, (pj, f, err)
