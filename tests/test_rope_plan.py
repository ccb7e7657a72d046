"""The turns per position that csa_rope_plan_init puts into a plan, against 60 decimal digits (host only)."""
import decimal

import pytest

import continuous_softmax_attention_gb300 as csa
from continuous_softmax_attention_gb300 import _lib as L

TWO_PI = decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194988918")


@pytest.fixture(scope="module", autouse=True)
def built():
    import os

    if not os.path.exists(L.LIB_PATH):
        from continuous_softmax_attention_gb300 import build

        build.build()


@pytest.mark.parametrize("base", [2.0, 10000.0, 500000.0, 1e7, 1e10, 1e15])
@pytest.mark.parametrize("n", [1, 2, 3, 12, 64, 127, 128])
def test_turns_per_position(base, n):
    plan = csa.RopeAxes(2 * n, (n,), base=base)._plan
    with decimal.localcontext() as c:
        c.prec = 60
        unit = decimal.Decimal(2) ** 64
        for i in range(n):
            exact = (-(decimal.Decimal(base).ln() * i / n)).exp() / TWO_PI * unit
            # rounded to nearest over 64 bits; before it (ln base + 4) 2^-64 relative where a long double has 64
            # bits: the exponent's rounding times ln base, the power's step, and a product
            off = abs(decimal.Decimal(plan.turn[i]) - exact)
            assert off <= decimal.Decimal("0.5") + exact * (decimal.Decimal(base).ln() + 4) / unit, (i, off)


def test_turns_of_a_base_below_one():
    # whole turns are dropped; the rest keeps what the larger number leaves
    plan = csa.RopeAxes(4, (2,), base=2.0 ** -20)._plan
    with decimal.localcontext() as c:
        c.prec = 60
        exact = decimal.Decimal(2) ** 10 / TWO_PI % 1
        assert abs(decimal.Decimal(plan.turn[1]) / 2 ** 64 - exact) <= decimal.Decimal(2) ** -64 * 2 ** 10 * 18
