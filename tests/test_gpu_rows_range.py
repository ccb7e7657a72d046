"""Drafted tokens with more than 16 rows per cached head (csa_decode_tree on tensor memory): scales, logits and queries far
from one another, over ranges of several tiles and several parts, against the CPU oracle."""
import numpy as np
import pytest
import torch

from continuous_softmax_attention_gb300 import device_status
from draft_util import KINDS
from test_gpu_tree import check, make, run

pytestmark = pytest.mark.gpu
ROWS = pytest.mark.parametrize("T,G", [(20, 1), (12, 4), (32, 4)], ids=["20 rows", "48 rows", "128 rows"])
EIGHT = pytest.mark.parametrize("kind", ["e4m3", "int8"])
KIND = pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])


def at(x, b, i):
    """Pages and slots of tokens i of sequence b."""
    i = torch.as_tensor(i)
    return torch.as_tensor(x["table"][b].astype(np.int64))[i // x["S"]], i % x["S"]


@EIGHT
@pytest.mark.parametrize("d", [64, 128, 256])
@ROWS
def test_scales_over_many_powers_of_two(kind, d, T, G):
    """Values' scales that rise, fall and jump within a range of tiles, and tiles of scale 0: the unit of the values follows."""
    n = 12000
    x = make(kind, [n] * 6, [T] * 6, T, G, 1, d, 64, seed=d + T)
    i, r = torch.arange(n), torch.randint(-12, 13, (n,), generator=torch.Generator().manual_seed(1)).float()
    for b, e in enumerate([torch.linspace(-60, 20, n), torch.linspace(20, -60, n), torch.where(i == n // 3, 30.0, -20.0),
                           torch.where(i % 50 == 0, -90.0, 0.0), torch.where(i < 400, -float("inf"), 0.0), r]):
        page, slot = at(x, b, i)
        x["scales"][page, :, slot, 1] *= torch.exp2(e)[:, None]
    for mode in (0, 1, 2):
        o, lse = run(x, mode)
        check(x, o, lse, mode, nodes={0, T - 1}, heads=(0, G - 1))
    assert device_status() == 0


@KIND
@pytest.mark.parametrize("d", [64, 128, 256])
@ROWS
def test_rising_and_falling_logits(kind, d, T, G):
    """Logits that rise, fall and leap while the rows of a range go by, by other factors for each query, and backwards."""
    n = 9000
    x = make(kind, [n] * 4, [T] * 4, T, G, 1, d, 64, seed=3)
    u = torch.randn(d, generator=torch.Generator().manual_seed(1))
    code = u.to(torch.bfloat16) if kind == "bf16" else (u / u.abs().max() * 100).to(KINDS[kind])
    factor = torch.as_tensor(np.random.default_rng(T).choice([1.0, -1.0, 0.5, -0.25, 0.125, 0.0], (4, G, T)), dtype=torch.float32)
    factor[:, :, 0], factor[:, :, T - 1] = 1.0, -1.0
    x["q"] = (factor[..., None] * u.to(torch.bfloat16).float()).to(torch.bfloat16)
    i, ramp = torch.arange(n), torch.linspace(-30, 30, n)
    unit = (code.float() @ u).item() / d ** 0.5  # logit of a row of scale 1
    for b, s in enumerate([ramp, ramp.flip(0), torch.where(i == 3777, 60.0, -ramp.abs()), torch.where(i // 700 % 2 == 0, 20.0, -20.0)]):
        page, slot = at(x, b, i)
        if kind == "bf16":
            x["k"][page, 0, slot] = (u * (s / unit)[:, None]).to(torch.bfloat16)
        else:
            x["k"].view(torch.uint8)[page, 0, slot] = torch.where((s >= 0)[:, None], code.view(torch.uint8), (-code.float()).to(KINDS[kind]).view(torch.uint8))
            x["scales"][page, 0, slot, 0] = s.abs() / unit
    o, lse = run(x, 0)
    check(x, o, lse, 0, nodes={0, 1, T // 2, T - 1}, heads=(0, G - 1))


@EIGHT
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("big", [2.0 ** 100, 2.0 ** -60, 3.0])
@ROWS
def test_queries_of_any_size(kind, d, big, T, G):
    """Queries and keys' scales far from 1 whose logits are ordinary, one element of a query far above the rest."""
    x = make(kind, [50, 1300], [T, T], T, G, 1, d, 32, seed=4)
    x["q"] = (x["q"].float() * big).to(torch.bfloat16)
    x["q"][:, :, ::2, 7] = 0
    x["q"][:, :, 1, 9] *= 32
    x["scales"][..., 0] /= big
    x["k0"] = (x["k0"].float() / big).to(torch.bfloat16)
    x["q"][0, 0, 3] = 0  # no direction at all
    for mode in (0, 2):
        o, lse = run(x, mode)
        check(x, o, lse, mode, nodes={0, 1, 3, T - 1}, heads=(0, G - 1))


@EIGHT
@pytest.mark.parametrize("d", [64, 128, 256])
@ROWS
def test_rows_that_are_not_numbers_show(kind, d, T, G):
    """A key or value before the draft that is not a number: its head's rows show it, in the weights or in the sums alone."""
    x = make(kind, [3000, 1500, 100, 700], [T] * 4, T, 3 * G, 3, d, 16, seed=22)
    want, wl = run(x, 0)
    y = dict(x, scales=x["scales"].clone())
    for b, i, head, which in ((0, 1717, 0, 0), (1, 5, 1, 1), (2, 99, 2, 0)):
        page, slot = at(y, b, [i])
        y["scales"][page, head, slot, which] = float("nan")
    o, lse = run(y, 0)
    for b, head, which in ((0, 0, 0), (1, 1, 1), (2, 2, 0)):
        mine = slice(head * G, head * G + G)
        assert torch.isnan(o[b, mine].float()).all() and bool(torch.isnan(lse[b, mine]).all()) == (which == 0)
        others = [h for h in range(3 * G) if h // G != head]
        assert torch.equal(o[b, others], want[b, others]) and torch.equal(lse[b, others], wl[b, others])
    assert torch.equal(o[3], want[3]) and torch.equal(lse[1], wl[1]) and device_status() == 0
