"""8-bit pools whose values' scales lie far apart (csa_decode_paged_q8, csa_decode_tree): what a row adds to the output counts
by its weight and its scale together, so a far larger scale of a row that has next to no weight costs the others nothing,
and neither does a small one of the rows that have it all."""
import numpy as np
import pytest
import torch

import oracle
from continuous_softmax_attention_gb300 import decode_paged, decode_tree, device_status
from draft_util import KINDS, random_pools, values
from paged_util import pages_of, rows_of, scattered

pytestmark = pytest.mark.gpu
EIGHT = pytest.mark.parametrize("kind", ["e4m3", "int8"])
INT = dict(dtype=torch.int32, device="cuda")


def patterns(n, g):
    """Logits (natural units) of n rows for a query of factor 1, and powers of two of their values' scales."""
    i, noise = torch.arange(n), torch.randn(n, generator=g)
    for lo, hi in ((n // 3, n // 2), (0, n // 3), (n - n // 4, n)):  # next to no weight, and scales 2^30 larger
        low = (i >= lo) & (i < hi)
        # the rows at the edges share intervals with the others
        yield torch.where(low, -60.0, noise), torch.where((i >= lo + 2 * (lo > 0)) & (i < hi - 2), 30.0, 0.0)
    yield torch.where(i % 97 < 5, -60.0, noise), torch.where(i % 97 == 2, 30.0, 0.0)    # single rows of that kind
    yield torch.where(i % 300 < 9, 60.0 + noise, noise), torch.where(i % 300 < 9, -30.0, 0.0)  # all weight on small values
    e = torch.linspace(-20, 40, n)
    yield -e * np.log(2), e  # every row adds as much as another
    yield -e.flip(0) * np.log(2), e.flip(0)
    for most in (40.0, -25.0):  # every row adds as much as another; as much as the sink at the ends
        e = most * torch.sin(np.pi * (i + 1) / (n + 1))
        yield -e * np.log(2), e
    yield 0.3 * noise, torch.where(i < n // 2, -float("inf"), 0.0)  # half of the rows are zeros


def make(kind, n, B, Hkv, d, S, seed):
    """B sequences of n rows, one pattern each; the keys of a head all lie on a direction u of their own."""
    g = torch.Generator().manual_seed(seed)
    P = B * pages_of(n, S) + 2
    k, v, scales = random_pools(P, Hkv, S, d, kind, g, spread=0.5)
    table = scattered([n] * B, S, P, seed)
    u = torch.randn(Hkv, d, generator=g).to(torch.bfloat16).float()
    code = (u / u.abs().amax(1, keepdim=True) * 100).to(KINDS[kind])
    i = torch.arange(n)
    for b, (logit, e) in enumerate(patterns(n, g)):
        page, slot = torch.as_tensor(table[b].astype(np.int64))[i // S], i % S
        for h in range(Hkv):
            unit = (code[h].float() @ u[h]).item() / d ** 0.5
            opposite = (-code[h].float()).to(KINDS[kind])
            k.view(torch.uint8)[page, h, slot] = torch.where((logit >= 0)[:, None], code[h].view(torch.uint8), opposite.view(torch.uint8))
            scales[page, h, slot, 0] = logit.abs() / unit
            scales[page, h, slot, 1] *= torch.exp2(e)
    k0, v0 = (torch.randn(Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    return dict(k=k, v=v, scales=scales, table=table, u=u, lens=[n] * B, S=S, k0=k0, v0=v0)


def queries(x, B, Hkv, G, T, seed):
    """Factors of the heads' directions: some look away from what the others look at."""
    f = torch.as_tensor(np.random.default_rng(seed).choice([1.0, -1.0, 0.5, 0.25], (B, Hkv, G, T)), dtype=torch.float32)
    f[..., 0, 0], f[..., G - 1, T - 1] = 1.0, (1.0 if G * T == 1 else -1.0)
    return (f[..., None] * x["u"][None, :, None, None]).to(torch.bfloat16).view(B, Hkv * G, T, -1)


def check(x, q, o, lse, rows, nodes, heads, mode=0, sign=1):
    """q, o [B, Hq, T, d]: row t of the chain that ends every sequence.

    Bound.  As draft_util.bounds, but by what the rows add: a weight is off by `rel` and by its rounding to fp16 (2^-11; with
    more than 16 rows 2.2e-4 more by the division of an interval, counted twice as each row has two), which moves o by as much
    of sum w |v| / sum w, the attention's output over |v|; the weights' sum by `rel` once more.  Below fp16's normal numbers a
    product of a weight and a scale is off by 2^-25 of the unit.  The unit makes 2^4 or more of the largest product's bound M,
    the largest power of a logit times the scales of its row and the neighbours; with more than 16 rows 2^-6 or more, where
    a tile's scales lie that close together.  So each row may be off by 2^-29 M, or 2^-19 M, times its largest code."""
    B, Hq, T, d = q.shape
    Hkv, scale = x["k"].shape[1], sign * d ** -0.5
    vk, vv = values(x["k"], x["v"], x["scales"])
    code = 448 if x["v"].dtype == KINDS["e4m3"] else 127
    o, lse = o.double().cpu().numpy(), lse.cpu().numpy()
    for b in range(B):
        n = x["lens"][b]
        k, v, s = (rows_of(t, x["table"][b], n, x["S"]) for t in (vk, vv, x["scales"].double()))
        for t in nodes:
            m = n - T + t + 1
            for h in heads:
                hk = h // (Hq // Hkv)
                qq = torch.zeros(1, 1, m, d, dtype=torch.float64)
                qq[0, 0, -1] = q[b, h, t].double()
                k0, v0 = x["k0"][hk:hk + 1].double(), x["v0"][hk:hk + 1].double()
                one = lambda f: oracle.forward_rows(qq, k[None, hk:hk + 1, :m], f(v[None, hk:hk + 1, :m]), [m - 1], k0=k0, v0=f(v0),  # noqa: E731
                                                    scale=scale, mode=mode)
                (ro, rl), (ao, _) = one(lambda y: y), one(torch.abs)
                a = scale * (k[hk, :m] @ q[b, h, t].double()).numpy()
                sink = 0.0 if mode == 0 else a[0] if mode == 1 else scale * (k0[0] @ q[b, h, t].double()).item()
                rel = (d + 8) * 2.0 ** -24 * max(np.abs(a).max(), abs(sink)) + 2.0 ** -16
                y = np.pad(s[hk, :m, 1].numpy(), 1)
                M = max((np.exp(a - rl[0]) * np.maximum(np.maximum(y[:-2], y[1:-1]), y[2:])).max(), np.exp(sink - rl[0]) * y[1])
                bound = 2.0 ** -8 * np.abs(ro[0]) + (2 * rel + 2.0 ** -11 + 2.0 ** -16 + (4.4e-4 if rows > 16 else 0.0)) * ao[0]
                bound = bound + m * (2.0 ** -19 if rows > 16 else 2.0 ** -29) * M * code
                err = np.abs(o[b, h, t] - ro[0])
                assert (err <= bound).all(), (b, h, t, float((err / bound).max()))
                assert abs(lse[b, h, t] - rl[0]) <= rel + 2.0 ** -22 * (1 + abs(rl[0])), (b, h, t, lse[b, h, t], rl[0])


@EIGHT
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 8, 16, 24])
@pytest.mark.parametrize("n,wide", [(700, False), (2500, True)], ids=["one kernel", "parts joined"])
def test_decode(kind, d, G, n, wide):
    x = make(kind, n, 10, 2, d, 16, seed=G)
    q = queries(x, 10, 2, G, 1, seed=d)
    for b in range(10) if not wide else [None]:  # alone a sequence has a cluster per head where the table is short
        part = slice(None) if wide else slice(b, b + 1)
        table = torch.as_tensor(x["table"])[part]
        if wide:
            table = torch.cat([table, torch.full((10, 2500), -1, dtype=torch.int32)], 1)
        o, lse = decode_paged(q[part, :, 0].contiguous().cuda(), x["k"].cuda(), x["v"].cuda(), table.contiguous().cuda(),
                              torch.tensor(x["lens"], **INT)[part], row_scales=x["scales"].cuda())
        one = dict(x, table=x["table"][part], lens=x["lens"][part])
        check(one, q[part], o[:, :, None], lse[:, :, None], G, [0], sorted({0, G - 1, 2 * G - 1}))
    assert device_status() == 0


@EIGHT
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(2, 1), (3, 4), (20, 1), (12, 4), (32, 4)])
def test_drafts(kind, d, T, G):
    x = make(kind, 5000, 10, 1, d, 64, seed=T)
    q = queries(x, 10, 1, G, T, seed=d)
    o, lse = decode_tree(q.cuda(), x["k"].cuda(), x["v"].cuda(), torch.as_tensor(x["table"]).cuda(), torch.tensor(x["lens"], **INT),
                         row_scales=x["scales"].cuda())
    check(x, q, o, lse, G * T, sorted({0, T // 2, T - 1}), sorted({0, G - 1}))
    assert device_status() == 0


@EIGHT
@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("T,G", [(1, 1), (1, 16), (3, 2), (20, 1), (12, 4), (16, 8)])
def test_sinks_and_a_negative_scale(kind, mode, T, G):
    """A copied sink, whose value is the first row's, and a given one; logits of the other sign."""
    x = make(kind, 3000, 10, 1, 128, 32, seed=T + G)
    q = queries(x, 10, 1, G, T, seed=mode)
    for sign in (1, -1):
        c = [t.cuda() for t in (q, x["k"], x["v"], torch.as_tensor(x["table"]), torch.tensor(x["lens"], dtype=torch.int32), x["k0"], x["v0"])]
        kw = dict(row_scales=x["scales"].cuda(), mode=mode, scale=sign * 128 ** -0.5)
        if T == 1:
            o, lse = (t[:, :, None] for t in decode_paged(c[0][:, :, 0].contiguous(), *c[1:], **kw))
        else:
            o, lse = decode_tree(*c[:5], None, *c[5:], **kw)
        check(x, q, o, lse, G * T, sorted({0, T - 1}), sorted({0, G - 1}), mode, sign)
    assert device_status() == 0
