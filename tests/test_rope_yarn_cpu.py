"""pkv_rope_inv_freq with YaRN over the whole ramp, against the published formula
in 50 digits: pair i is kept below floor(c(beta_fast)), stretched above
ceil(c(beta_slow)), and between them mixed in proportion to its index, with
c(beta) = R ln(trained / (2 pi beta)) / (2 ln theta)."""
from decimal import Decimal, getcontext
import math

import pytest

import paged_kv_decode_13_gb300 as pkv

getcontext().prec = 50
PI = Decimal("3.14159265358979323846264338327950288419716939937511")


@pytest.mark.parametrize("rot", [32, 64, 128, 256])
@pytest.mark.parametrize("theta,factor,trained,fast,slow", [(10000.0, 16.0, 4096.0, 32.0, 1.0), (500000.0, 8.0, 8192.0, 32.0, 1.0), (1e6, 4.0, 32768.0, 32.0, 1.0),
                                                            (10000.0, 40.0, 2048.0, 64.0, 2.0), (10000.0, 2.0, 100.0, 32.0, 1.0)])
def test_ramp(rot, theta, factor, trained, fast, slow):
    got, m = pkv.rope_inv_freq(rot, theta, "yarn", factor, trained, fast, slow)
    T, F = Decimal(theta), Decimal(factor)

    def c(beta):
        return Decimal(rot) * (Decimal(trained) / (2 * PI * Decimal(beta))).ln() / (2 * T.ln())

    lo, hi = max(math.floor(c(fast)), 0), min(math.ceil(c(slow)), rot - 1)
    mixed = 0
    for i in range(rot // 2):
        f = (-Decimal(2 * i) / Decimal(rot) * T.ln()).exp()
        r = min(max((Decimal(i) - lo) / Decimal(max(hi - lo, 0) or "0.001"), Decimal(0)), Decimal(1))
        want = f / F * r + f * (1 - r)
        mixed += 0 < r < 1
        # pow to 2^-52 of its exponent's error 2^-53 * |ln f| < 2^-49, and four roundings
        assert abs(Decimal(float(got[i])) - want) <= want * Decimal(2) ** -47, i
    assert mixed >= 2 or trained == 100.0
    assert abs(m - (0.1 * math.log(factor) + 1.0)) < 1e-15 * 8
