"""How far the frequencies that a Rotary holds, in 2^-64 of a circle a position, are from the formula: against 60 decimal digits.
A frequency f of at most a radian is computed in doubles, half a step of which is 2^-53 of it. The power is off by less than two
of these, a larger base by two more at most, a scaling's sum and product by five, 2 pi and the division by two: at most nine are
together, and 9 * 2^-53 / (2 pi) < 2^-52."""
import math
from decimal import Decimal, localcontext

import pytest

import sparse_mixture_experts_moe_gb300 as moe

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def frequencies(R, base, scaling, factor, length):
    """Radians a position of each pair."""
    b, s = Decimal(base), Decimal(factor)
    if scaling == "base":
        b *= (s.ln() * R / (R - 2)).exp()

    def pair(turns):
        return R * (length / (2 * PI * turns)).ln() / (2 * b.ln())
    for p in range(R // 2):
        f, kept = (b.ln() * -2 * p / R).exp(), Decimal(1)
        if scaling == "linear":
            kept = Decimal(0)
        elif scaling == "turns":
            kept = min(Decimal(1), max(Decimal(0), (length * f / (2 * PI) - 1) / 3))
        elif scaling == "pairs":
            first, last = max(0, math.floor(pair(32))), min(R - 1, math.ceil(pair(1)))
            kept = Decimal(1) if p <= first else Decimal(0) if p >= last else Decimal(last - p) / (last - first)
        yield f * (kept + (1 - kept) / s) if scaling in ("linear", "turns", "pairs") else f


@pytest.mark.parametrize("scaling", [None, "linear", "base", "turns", "pairs"])
@pytest.mark.parametrize("base", [1.5, 1000.0, 10000.0, 500000.0])
@pytest.mark.parametrize("R", [2, 6, 64, 80, 128, 256])
def test_frequencies(R, base, scaling):
    if scaling == "base" and R == 2:
        pytest.skip("refused")
    rope = moe.Rotary(max(8, -(-R // 8) * 8), rotary_dim=R, base=base, scaling=scaling, factor=1.0 if scaling is None else 7.3,
                      original_len=4096)
    with localcontext() as c:
        c.prec = 60
        for p, f in enumerate(frequencies(R, base, scaling, 7.3, 4096)):
            assert abs(Decimal(rope._c.turns[p]) / 2 ** 64 - f / (2 * PI)) < Decimal(2) ** -52
