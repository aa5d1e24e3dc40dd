"""The frequencies of a rotation plan are doubles, and they bound the angle at far positions: against
50-digit arithmetic they are within 2^-24 turns over 2^31 positions (a frequency of 1 / (2 pi), the highest,
rounds at 2^-56, and the power and the division before it at a few times that)."""
from decimal import Decimal, getcontext

import pytest

import block_masked_window_b200 as bmw

PI = Decimal("3.14159265358979323846264338327950288419716939937510582")


@pytest.mark.parametrize("base", [10000.0, 1e6])
@pytest.mark.parametrize("rotary", [64, 128, 256])
def test_turns(base, rotary):
    getcontext().prec = 50
    plan = bmw.RopePlan.make(rotary, base=base)
    log = Decimal(base).ln()
    worst = max(abs(Decimal(plan.turns[i]) - (-log * 2 * i / rotary).exp() / (2 * PI)) for i in range(rotary // 2))
    assert worst * 2 ** 31 <= Decimal(2) ** -24
    assert worst * 2 ** 31 > Decimal(2) ** -31      # more than the product and its reduction add
