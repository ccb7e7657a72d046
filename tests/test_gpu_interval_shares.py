"""How an interval's integral is divided between its two rows with more than 16 rows per cached head (csa_decode_tree),
where the formula changes between a series and quotients."""
import numpy as np
import pytest
import torch

import oracle
from continuous_softmax_attention_gb300 import decode_tree
from paged_util import scattered

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [32, 64, 128])
def test_an_interval_is_divided_within_its_bound(rows):
    """Logits in turn 0 and x above a common level, values in turn -1 and 1: every interval is the same or its mirror, so
    an error of the division adds up.  One row before them is higher, so that both exponentials of an interval are rounded.

    Bound.  Keys are at most two powers of two, queries multiples of 2^-14 below 8: products and their sums are exact, and
    a logit is rounded with the scale, its factor and its maximum, 4 * 2^-24 of the largest in all, A; integrals 2^-16 and
    weights as two bf16 numbers 2^-16.  A share is off by at most 2.2e-4 of itself and the other by as much absolutely.
    Shares are nearly halves of an interval, and values 2 apart: o is off by at most 2.3e-4, and 2^-8 |o| for its rounding."""
    n, d, S = 6000, 64, 64
    r = np.random.default_rng(rows)
    k = torch.zeros(n + 1, d)
    k[1::2, 0], k[1::2, 1] = 1, 2.0 ** -7
    k[1:, 2] = 1
    k[0, 3] = 1
    v = torch.where(torch.arange(n + 1) % 2 == 1, 1.0, -1.0)[:, None].repeat(1, d)
    v[0] = 0  # o is small, and so its rounding
    P = -(-(n + 1) // S)
    table = scattered([n + 1], S, P, 0)
    kp, vp = (torch.zeros(P, 1, S, d, dtype=torch.bfloat16) for _ in range(2))
    for pool, x in ((kp, k), (vp, v)):
        for j in range(P):
            pool[table[0, j], 0, :len(x[j * S:(j + 1) * S])] = x[j * S:(j + 1) * S].to(torch.bfloat16)
    worst = 0.0
    for call in range(4):
        q = torch.zeros(rows, d, dtype=torch.float64)
        x = np.exp2(r.uniform(np.log2(0.03), np.log2(0.25), rows))
        q[:, 0] = torch.as_tensor(np.floor(x * 2 ** 9) / 2 ** 9)
        q[:, 1] = torch.as_tensor(r.integers(0, 128, rows) / 2.0 ** 7)
        q[:, :2] *= torch.as_tensor(r.choice([-1.0, 1.0], rows))[:, None]
        q[:, 2] = torch.as_tensor(r.integers(-64, 65, rows) / 64.0)
        q[:, 3] = torch.as_tensor(r.integers(128, 256, rows) / 32.0)
        assert torch.equal(q, q.to(torch.bfloat16).double())
        INT = dict(dtype=torch.int32, device="cuda")
        o, _ = decode_tree(q.view(1, rows, 1, d).to(torch.bfloat16).cuda(), kp.cuda(), vp.cuda(), torch.as_tensor(table).cuda(),
                           torch.tensor([n + 1], **INT), scale=1.0)
        o = o[0, :, 0, 0].double().cpu().numpy()
        for h in range(rows):
            qq = torch.zeros(1, 1, n + 1, d, dtype=torch.float64)
            qq[0, 0, n] = q[h]
            ref, _ = oracle.forward_rows(qq, k.double()[None, None], v.double()[None, None], [n], scale=1.0)
            A = (k.double() @ q[h]).abs().max().item()
            bound = 2.0 ** -8 * abs(ref[0, 0]) + 2.3e-4 + 2 * (4 * 2.0 ** -24 * A + 2.0 ** -16) + 2.0 ** -16
            worst = max(worst, abs(o[h] - ref[0, 0]) / bound)
    assert worst <= 1, worst
