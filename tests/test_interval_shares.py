"""The division of an interval's integral between its two rows, as csa_rows.cuh forms it in fp32, against the formula in
64 bits: its bounds, with exponentials that are off by the most that ex2.approx may be."""
import os
import re

import numpy as np
import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "continuous_softmax_attention_gb300", "csrc",
                      "csa_rows.cuh")
F = np.float32
LN2 = F(0.6931471805599453)


def border():
    """Where the formula changes from a series to quotients, log2 units."""
    text = open(SOURCE).read()
    name = re.search(r"s0 = fabsf\(x0\) < ([\w.]+)", text).group(1)
    return float((re.search(rf"{name} = ([\d.]+)f;", text).group(1) if name[0] == "k" else name.rstrip("f")))


def fma(a, b, c):
    return (a.astype(np.float64) * np.float64(b) + np.asarray(c, np.float64)).astype(F)  # products of 48 bits


def shares(u0, u1, e0, e1, at):
    """(left, right) times (ln 2)^2 as the kernel forms them, the exponentials off by e0 and e1."""
    p0, p1 = ((np.exp2(u.astype(np.float64)) * (1 + e)).astype(F) for u, e in ((u0, e0), (u1, e1)))
    x = u0 - u1
    near = np.abs(x) < F(at)
    inv = F(1) / np.where(near, F(1), x)
    g = np.where(near, F(1), F(-1))
    S = fma(p1, g, p0) * np.where(near, fma(x * x, -LN2 * LN2 * LN2 / F(24), F(0.5) * LN2), inv)
    R = fma(p0, np.where(near, F(0.5) * LN2, -LN2), S) * np.where(near, -LN2 / F(3), inv)
    return -R, fma(S, LN2, R)


def phi2(x):
    small = np.abs(x) < 0.1
    y = np.where(small, 1.0, x)
    series = sum(x ** n / float(np.prod(np.arange(1.0, n + 3))) for n in range(10))
    return np.where(small, series, (np.expm1(y) - y) / y ** 2)


@pytest.mark.parametrize("errors", [(0.0, 0.0), (2.0 ** -22, -(2.0 ** -22)), (-(2.0 ** -22), 2.0 ** -22)])
def test_shares_and_integrals_are_within_their_bounds(errors):
    """A share within 2.2e-4 of itself and the integral within 2^-16.8, both of what csa_rows.cuh states."""
    r = np.random.default_rng(0)
    n, at = 200000, border()
    for lo, hi in ((1e-4, at), (at, 1.1 * at), (at, 20.0)):
        u0 = r.uniform(-16, 6, n).astype(F)
        u1 = (u0 + np.exp(r.uniform(np.log(lo), np.log(hi), n)) * r.choice([-1, 1], n)).astype(F)
        left, right = (t.astype(np.float64) / np.log(2) ** 2 for t in shares(u0, u1, *errors, at))
        X = (u1.astype(np.float64) - u0) * np.log(2)
        want_l, want_r = np.exp2(u0.astype(np.float64)) * phi2(X), np.exp2(u1.astype(np.float64)) * phi2(-X)
        alike = np.abs(X) < 1  # a share far below the other takes that one's error
        assert np.abs(left / want_l - 1)[alike].max() <= 2.2e-4 and np.abs(right / want_r - 1)[alike].max() <= 2.2e-4, (lo, hi)
        assert np.abs((left + right) / (want_l + want_r) - 1).max() <= 2.0 ** -16.8, (lo, hi)
