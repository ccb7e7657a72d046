"""Rows of 8 bits read back as bf16: the product of code and scale is rounded once (csa_cache_read)."""
import numpy as np
import pytest
import torch

from continuous_softmax_attention_gb300 import cache_read
from draft_util import KINDS

pytestmark = pytest.mark.gpu


def to_bf16(x):
    """64-bit values to the nearest of 8 bits, ties to even."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


@pytest.mark.parametrize("d", [128, 127])  # eight codes at a time, and one
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_a_product_is_rounded_once(kind, d):
    """Scales of 24 bits for which a code's product, rounded to fp32, lies in the middle between two bf16 numbers while the
    product itself does not: rounded twice, it would end on the other side of it.  A product has 31 bits: exact in 64."""
    codes = torch.arange(256, dtype=torch.uint8).view(KINDS[kind])
    value = codes.double().numpy() if kind == "int8" else codes.float().double().numpy()
    r = np.random.default_rng(1)
    # middles between two bf16 numbers, as fp32 quotients by a code that make a product next to it and not in it
    odd = np.array([c for c in (3, 5, 7, 9, 11, 13, 15, 99, 127) if c in value], np.float64)
    code, middle = r.choice(odd, 1000), (257 + 2 * r.integers(0, 128, 1000)) * np.exp2(r.integers(-60, 60, 1000))
    s = (middle / code).astype(np.float32)
    exact = code * s.astype(np.float64)
    twice = to_bf16(exact.astype(np.float32).astype(np.float64)) != to_bf16(exact)
    rows = s[twice][:64]
    assert len(rows) == 64
    S, P = 16, -(-2 * len(rows) // 16)
    k = torch.zeros(P, 1, S, d, dtype=torch.uint8)
    scales = torch.ones(P, 1, S, 2)
    finite = torch.as_tensor(np.flatnonzero(np.isfinite(value)))
    for i in range(2 * len(rows)):  # half of the codes in a row of its own each
        of = finite[i % 2::2][:d] if d < len(finite) // 2 else finite[i % 2::2]
        k[i // S, 0, i % S, :len(of)] = codes.view(torch.uint8)[of]
        scales[i // S, 0, i % S] = float(rows[i // 2])
    pool = k.view(KINDS[kind])
    table, n = torch.arange(P, dtype=torch.int32).view(1, P), 2 * len(rows)
    got, _ = cache_read(pool.cuda(), pool.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), n, row_scales=scales.cuda())
    want = to_bf16(pool.view(1, P * S, d)[:, :n].float().double().numpy() * scales.view(1, P * S, 2)[:, :n, :1].double().numpy())
    assert np.array_equal(got[:, 0].double().cpu().numpy(), want)
