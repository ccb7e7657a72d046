"""Angles of the rotary positions on isolated pairs, where sine and cosine come out unmixed, against
angles formed in 60 decimal digits and with bounds relative to each value."""
import decimal
import math

import numpy as np
import pytest
import torch

from continuous_softmax_attention_gb300 import RopeAxes, rope, rope_backward

pytestmark = pytest.mark.gpu

POSITIONS = [0, 1, -1, 2, -3, 1000, -1000, 2 ** 20 + 1, -(2 ** 24) - 1, 2 ** 31 - 1, -2 ** 31]
TWO_PI = decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194988918")


def turned(p, i, n, base):
    """(sine, cosine, turns per position) of pair i at position p: the angle's distance to the nearest
    quarter of a turn in decimals, the functions of that distance in double."""
    with decimal.localcontext() as c:
        c.prec = 60
        per = (-(decimal.Decimal(base).ln() * i / n)).exp() / TWO_PI
        quarters = 4 * p * per
        near = quarters.to_integral_value(decimal.ROUND_HALF_EVEN)
        a, q = float((quarters - near) * TWO_PI / 4), int(near) % 4
    s, c = math.sin(a), math.cos(a)
    return [(s, c), (c, -s), (-s, -c), (-c, s)][q] + (float(per),)


@pytest.mark.parametrize("base", [10000.0, 500000.0, 1e7, 1e10])
@pytest.mark.parametrize("adjacent", [False, True])
def test_sine_and_cosine_of_every_angle(base, adjacent):
    n = 32
    plan = RopeAxes(2 * n, (n,), base=base, adjacent=adjacent)
    pos = torch.tensor(POSITIONS, dtype=torch.int32).cuda()
    x = torch.zeros(1, 1, len(POSITIONS), 2 * n, device="cuda")
    second = slice(1, None, 2) if adjacent else slice(n, None)
    first = slice(0, None, 2) if adjacent else slice(0, n)
    x[..., second] = 1.0  # (0, 1) becomes (-sin, cos), without a rounding
    y = rope(x, None, pos, plan)[0][0, 0].double().cpu().numpy()
    ref = np.array([[turned(p, i, n, base) for i in range(n)] for p in POSITIONS])
    p = np.abs(np.array(POSITIONS, np.float64))[:, None]
    # With u = 2^-24.  The distance x to the nearest quarter turn is the sum of two rounded words, 2u relative, which
    # neither function makes larger within an eighth of a turn (cosine: 0.8 times).  Sine: the last sum rounds by u, the
    # terms behind pi x, an eighth of it, by 5u of theirs; cosine: the last sum by 0.7u, the terms behind 1, at most 0.42
    # of the result, by 3u of theirs.  Together below 4u.  The turns per position are off by 2^-65 for the rounding to
    # 64 bits and by (ln base + 4) 2^-64 relative, ln base < 24.
    off = 2 * math.pi * p * (2.0 ** -65 + 28 * 2.0 ** -64 * ref[..., 2])
    for got, want in ((-y[:, first], ref[..., 0]), (y[:, second], ref[..., 1])):
        err, most = np.abs(got - want), 4 * 2.0 ** -24 * np.abs(want) + off
        assert (err <= most).all(), float((err / np.maximum(most, 1e-300)).max())


@pytest.mark.parametrize("d,sections,dtype", [(128, (16, 24, 24), torch.float32), (80, (10, 10), torch.bfloat16), (63, (5, 9), torch.float32)])
def test_opposite_positions_turn_by_opposite_angles(d, sections, dtype):
    plan = RopeAxes(d, sections, base=1e6)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 3, 40, d, generator=g).to(dtype).cuda()
    pos = torch.randint(-2 ** 31 + 1, 2 ** 31, (len(sections), 2, 40), generator=g, dtype=torch.int64).int().cuda()
    pos[:, 0] = torch.arange(40, dtype=torch.int32, device="cuda")
    assert torch.equal(rope(x, None, -pos, plan)[0], rope_backward(x, None, pos, plan)[0])
