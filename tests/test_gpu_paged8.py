"""Decode step over 8-bit pages (csa_decode_paged_q8) against the CPU oracle on the
values that the codes and scales stand for."""
import numpy as np
import pytest
import torch

import oracle
from continuous_softmax_attention_gb300 import (CsaError, RopeAxes, cache_append, decode_paged, decode_paged_workspace_bytes,
                                                device_status)
from draft_util import KINDS, bounds8, random_pools, values
from paged_util import pages_of, rows_of, scattered

pytestmark = pytest.mark.gpu
EIGHT = pytest.mark.parametrize("kind", ["e4m3", "int8"])
FORMS = pytest.mark.parametrize("wide", [False, True], ids=["one kernel", "parts joined"])
INT = dict(dtype=torch.int32, device="cuda")


def make(kind, lens, Hq, Hkv, d, S, seed, spare=3, wide=False, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    P = sum(pages_of(n, S) for n in lens) + spare
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    k, v, scales = random_pools(P, Hkv, S, d, kind, g, spread)
    return dict(q=bf(len(lens), Hq, d), k=k, v=v, scales=scales, k0=bf(Hkv, d), v0=bf(Hkv, d), lens=list(lens),
                table=scattered(lens, S, P, seed, M=pages_of(40000, S) if wide else None))


def dev(x):
    c = {n: t.cuda() for n, t in x.items() if torch.is_tensor(t)}
    return dict(c, table=torch.as_tensor(x["table"]).cuda(), lens=torch.tensor(x["lens"], **INT))


def call(c, mode=0, scale=None, **kw):
    return decode_paged(c["q"], c["k"], c["v"], c["table"], c["lens"], c["k0"], c["v0"], row_scales=c["scales"], mode=mode, scale=scale, **kw)


def run(x, mode=0, scale=None, **kw):
    o, lse = call(dev(x), mode, scale, **kw)
    torch.cuda.synchronize()
    return o, lse


def check(x, o, lse, S, mode, scale, only=None, heads=None):
    B, Hq, d = x["q"].shape
    Hkv = x["k"].shape[1]
    vk, vv = values(x["k"], x["v"], x["scales"])
    o, lse = o.double().cpu().numpy(), lse.cpu().numpy()
    for b in range(B) if only is None else only:
        n = x["lens"][b]
        if n == 0:
            assert (o[b] == 0).all() and np.isneginf(lse[b]).all()
            continue
        k, v = (rows_of(t, x["table"][b], n, S) for t in (vk, vv))
        for h in range(Hq) if heads is None else heads:
            hk = h // (Hq // Hkv)
            q = torch.zeros(1, 1, n, d, dtype=torch.float64)
            q[0, 0, n - 1] = x["q"][b, h].double()
            ro, rl = oracle.forward_rows(q, k[None, hk:hk + 1], v[None, hk:hk + 1], [n - 1], k0=x["k0"][hk:hk + 1].double(),
                                         v0=x["v0"][hk:hk + 1].double(), scale=scale, mode=mode)
            first = {0: (k[hk, :1] * 0, v[hk, :1] * 0), 1: (k[hk, :1], v[hk, :1]),
                     2: (x["k0"][hk:hk + 1].double(), x["v0"][hk:hk + 1].double())}[mode]
            bo, bl = bounds8(x["q"][b, h].double(), torch.cat([first[0], k[hk]]), torch.cat([first[1], v[hk]]), ro[0], rl[0], scale)
            err = np.abs(o[b, h] - ro[0])
            assert (err <= bo).all(), (b, h, n, float(err.max()), float((err / bo).max()))
            assert abs(lse[b, h] - rl[0]) <= bl, (b, h, n, float(lse[b, h]), float(rl[0]), bl)


EDGES = [1, 2, 3, 4, 5, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 0, 127, 128, 129, 200]


@EIGHT
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("S", [8, 16, 24, 64])
@FORMS
def test_lengths_around_every_edge(kind, d, mode, S, wide):
    x = make(kind, EDGES, 2, 1, d, S, seed=d + S + mode, wide=wide)
    o, lse = run(x, mode)
    check(x, o, lse, S, mode, d ** -0.5)


@EIGHT
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("Hq", [1, 3, 4, 7])
@FORMS
def test_edges_with_any_number_of_copies_of_the_heads(kind, d, mode, Hq, wide):
    """Eight rows hold a head eight times, two four times, up to four twice and more once."""
    x = make(kind, EDGES + [1000], Hq, 1, d, 16, seed=Hq + mode, wide=wide)
    o, lse = run(x, mode)
    check(x, o, lse, 16, mode, d ** -0.5)


@EIGHT
@pytest.mark.parametrize("Hq", [1, 2, 4, 6])
def test_a_head_does_not_see_the_others(kind, Hq):
    """Heads of a group share products: one with NaN for a query, or with far larger logits, leaves the others right.  Not
    bit for bit: all heads of a product raise the maximum that their weights are relative to when one of them passes its
    own, and a sum times 2^x, x not whole, is another fp32 number than the sum of the terms times it (each within 2^-22, of
    which `bounds8` allows (d + 8) 2^-24 A + 2^-16)."""
    x = make(kind, [700, 33], Hq, 1, 128, 16, seed=4, wide=True)
    for h in range(Hq):
        for factor in (float("nan"), 64.0):
            y = dict(x, q=x["q"].clone())
            y["q"][:, h] *= factor
            o, lse = run(y, 0)
            check(x, o, lse, 16, 0, 128 ** -0.5, heads=[i for i in range(Hq) if i != h])
            assert torch.isnan(o[:, h].float()).all() if factor != factor else torch.isfinite(o[:, h].float()).all()


@EIGHT
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 2), (10, 2), (16, 1), (9, 1), (17, 1), (33, 11)])
@FORMS
def test_head_groups(kind, d, Hq, Hkv, wide):
    x = make(kind, [5, 333, 0, 40, 1, 1500], Hq, Hkv, d, 32, seed=Hq, wide=wide)
    o, lse = run(x, 2)
    check(x, o, lse, 32, 2, d ** -0.5)


@EIGHT
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.125, 1.0, 4.0, -0.5, 0.0])
@FORMS
def test_logit_ranges(kind, d, scale, wide):
    x = make(kind, [1, 2, 30, 300, 700], 4, 2, d, 16, seed=17, wide=wide)
    o, lse = run(x, 1, scale)
    check(x, o, lse, 16, 1, scale)


@EIGHT
@pytest.mark.parametrize("Hq", [2, 12])
@FORMS
def test_scales_over_many_powers_of_two(kind, Hq, wide):
    """Scales that rise, fall and jump within a sequence: the unit of the values follows them."""
    lens = [700, 700, 700, 700, 40]
    x = make(kind, lens, Hq, 1, 128, 16, seed=21, wide=wide)
    i = torch.arange(700)
    rise = [torch.linspace(-60, 20, 700), torch.linspace(20, -60, 700), torch.where(i == 333, 30.0, -20.0), torch.where(i % 50 == 0, -90.0, 0.0), i[:40] * 0 - 95.0]
    for b, r in enumerate(rise):
        for t in range(lens[b]):
            x["scales"][x["table"][b, t // 16], :, t % 16, 1] = 2.0 ** float(r[t])
    x["scales"][..., 1][x["scales"][..., 1] < 2.0 ** -89] *= 1.3
    o, lse = run(x, 1)
    check(x, o, lse, 16, 1, 128 ** -0.5)


@EIGHT
@FORMS
def test_rising_and_falling_logits(kind, wide):
    n, d = 500, 128
    x = make(kind, [n, n, n], 1, 1, d, 16, seed=3, wide=wide)
    u = torch.randn(d, generator=torch.Generator().manual_seed(1))
    ramp = torch.linspace(-30, 30, n)
    shapes = [ramp, ramp.flip(0), torch.where(torch.arange(n) == 377, torch.tensor(60.0), -ramp.abs())]
    x["q"][:] = u.to(torch.bfloat16)
    code = (u / u.abs().max() * 100).to(KINDS[kind])
    for b, s in enumerate(shapes):
        for i in range(n):
            page, slot = x["table"][b, i // 16], i % 16
            x["k"][page, 0, slot] = code if s[i] >= 0 else (-code.float()).to(KINDS[kind])
            x["scales"][page, 0, slot, 0] = s[i].abs() / (code.float() @ u) * d ** 0.5
    o, lse = run(x, 0)
    check(x, o, lse, 16, 0, d ** -0.5)


@EIGHT
@pytest.mark.parametrize("big", [2.0 ** 100, 2.0 ** -60, 3.0])
def test_queries_of_any_size(kind, big):
    """Queries and scales far from 1 whose logits are ordinary, one element of a query far above the rest."""
    x = make(kind, [50, 600], 10, 2, 64, 16, seed=4)
    x["q"] = (x["q"].float() * big).to(torch.bfloat16)
    x["q"][:, ::2, 7] = 0
    x["q"][:, 1, 9] *= 32
    x["scales"][..., 0] /= big
    x["k0"] = (x["k0"].float() / big).to(torch.bfloat16)
    for mode in (0, 2):
        o, lse = run(x, mode)
        check(x, o, lse, 16, mode, 64 ** -0.5)
    x["q"][0, 3] = 0  # no direction at all
    o, lse = run(x, 0)
    check(x, o, lse, 16, 0, 64 ** -0.5)


@EIGHT
@pytest.mark.parametrize("d,S,Hq,Hkv", [(128, 64, 8, 2), (64, 256, 16, 2), (256, 16, 4, 4), (64, 8, 2, 1)])
def test_long_and_ragged(kind, d, S, Hq, Hkv):
    x = make(kind, [20011, 1, 0, 4097, 300, 12000], Hq, Hkv, d, S, seed=d)
    o, lse = run(x, 0)
    check(x, o, lse, S, 0, d ** -0.5)


@EIGHT
def test_many_short_sequences(kind):
    lens = [int(n) for n in np.random.default_rng(5).integers(0, 90, 300)]
    x = make(kind, lens, 8, 4, 128, 16, seed=6)
    o, lse = run(x, 1)
    check(x, o, lse, 16, 1, 128 ** -0.5, only=range(0, 300, 7))


@EIGHT
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq", [2, 24])
@FORMS
def test_pages_hold_anything_behind_the_last_token(kind, d, Hq, wide):
    lens, S = [1, 17, 100, 0, 129, 2040], 8
    x = make(kind, lens, Hq, 2, d, S, seed=d + Hq, wide=wide)
    want, wl = run(x, 0)
    held = set()
    for b, n in enumerate(lens):
        ids = x["table"][b, :pages_of(n, S)]
        held.update(ids.tolist())
        if n % S:
            for t in ("k", "v"):  # 127 is NaN of e4m3
                x[t].view(torch.uint8)[ids[-1], :, n % S:] = 127
            x["scales"][ids[-1], :, n % S:] = torch.tensor([float("nan"), float("inf")])
    rest = [p for p in range(x["k"].shape[0]) if p not in held]
    x["k"].view(torch.uint8)[rest], x["scales"][rest] = 255, float("nan")
    need = decode_paged_workspace_bytes(len(lens), Hq, 2, d)
    for fill in (255, 0, 127):
        o, lse = run(x, 0, workspace=torch.full((max(need, 16),), fill, dtype=torch.uint8, device="cuda"))
        assert torch.equal(o, want) and torch.equal(lse, wl)
    assert device_status() == 0


@EIGHT
@FORMS
def test_rows_that_are_not_numbers_show(kind, wide):
    x = make(kind, [40, 700, 30], 4, 2, 128, 16, seed=22, wide=wide)
    x["scales"][x["table"][0, 1], 0, 5, 0] = float("nan")   # a key of head 0
    x["scales"][x["table"][1, 20], 1, 5, 1] = float("nan")  # a value of head 1
    o, lse = run(x, 0)
    assert torch.isnan(o[0, :2].float()).all() and torch.isnan(lse[0, :2]).all() and torch.isnan(o[1, 2:].float()).all()
    assert torch.isfinite(o[0, 2:].float()).all() and torch.isfinite(o[1, :2].float()).all() and torch.isfinite(lse[1]).all() and torch.isfinite(o[2].float()).all()


@EIGHT
@FORMS
def test_bad_lengths_and_pages_are_reported(kind, wide):
    S, d = 16, 128
    x = make(kind, [100, 40, 60, 70, 0], 4, 2, d, S, seed=11, wide=wide)
    x["lens"][1] = x["table"].shape[1] * S + 1
    x["lens"][4] = -3
    x["table"][2, 1] = x["k"].shape[0]
    o, lse = run(x, 0)
    assert device_status() == -1 and device_status() == 0
    for b in (1, 2, 4):
        assert torch.isnan(o[b].float()).all() and torch.isnan(lse[b]).all()
    check(x, o, lse, S, 0, d ** -0.5, only=(0, 3))


@EIGHT
def test_no_pool(kind):
    e = torch.zeros(0, 2, 16, 64, device="cuda").to(KINDS[kind])
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(0, 2, 16, 2, device="cuda")
    table = torch.full((3, 2), -1, **INT)
    o, lse = decode_paged(q, e, e, table, torch.zeros(3, **INT), row_scales=s)
    assert not o.any() and torch.isneginf(lse).all() and device_status() == 0
    o, lse = decode_paged(q, e, e, table, torch.tensor([0, 5, 40], **INT), row_scales=s)
    assert not o[0].any() and torch.isnan(o[1:].float()).all() and device_status() == -1


def test_pages_beyond_32_bits():
    """Pools of 4.7e9 codes; the sequences' pages lie at both ends."""
    P, Hkv, S, d = 72000, 4, 64, 256
    lens = [300, 1000, 64]
    x = make("int8", lens, 8, Hkv, d, S, seed=31)
    far = {p: (P - 1 - p if p % 2 else p) for p in range(x["k"].shape[0])}
    k, v = (torch.zeros(P, Hkv, S, d, dtype=torch.int8, device="cuda") for _ in range(2))
    scales = torch.zeros(P, Hkv, S, 2, device="cuda")
    for p, f in far.items():
        k[f], v[f], scales[f] = x["k"][p].cuda(), x["v"][p].cuda(), x["scales"][p].cuda()
    table = torch.as_tensor([[far.get(int(e), -1) for e in row] for row in x["table"]], dtype=torch.int32).cuda()
    o, lse = decode_paged(x["q"].cuda(), k, v, table, torch.tensor(lens, **INT), row_scales=scales)
    check(x, o, lse, S, 0, d ** -0.5)


@EIGHT
@FORMS
def test_two_streams_and_a_graph_with_other_lengths(kind, wide):
    x = make(kind, [500, 300, 20], 4, 2, 64, 16, seed=14, wide=wide)
    c = dev(x)
    o, lse = call(c)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for i in range(12):
        got.append(call(c, stream=streams[i % 3]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) and torch.equal(lse, b) for a, b in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = call(c)
    for now in ([500, 300, 20], [1, 299, 0], [480, 1, 17]):
        c["lens"].copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        x["lens"] = now
        check(x, o, lse, 16, 0, 64 ** -0.5)


@EIGHT
def test_near_the_step_over_bf16_pages(kind):
    """The same tokens appended to bf16 and to 8-bit pools: outputs as far apart as the codes' rounding."""
    g = torch.Generator().manual_seed(5)
    B, H, T, d, S = 2, 2, 150, 128, 16
    k, v = torch.randn(2, B, H, T, d, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(B, 4, d, generator=g).to(torch.bfloat16).cuda()
    table = torch.arange(B * 10, **INT).view(B, 10)
    lens = torch.full((B,), T, **INT)
    plan = RopeAxes(d, (d // 2,))
    wide = [torch.zeros(20, H, S, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    narrow = [torch.zeros(20, H, S, d, device="cuda").to(KINDS[kind]) for _ in range(2)]
    scales = torch.zeros(20, H, S, 2, device="cuda")
    cache_append(k, v, *wide, table, lens, rope=plan)
    cache_append(k, v, *narrow, table, lens, rope=plan, row_scales=scales)
    a, la = decode_paged(q, *wide, table, lens)
    b, lb = decode_paged(q, *narrow, table, lens, row_scales=scales)
    # a code is off by 2^-4 of its value (e4m3) or 1/254 of the row's largest; errors of 128 columns and 150 rows add as squares
    tol = 0.1 if kind == "e4m3" else 0.03
    assert ((a - b).float().norm() / a.float().norm()).item() < tol and (la - lb).abs().max().item() < tol


def test_refusals():
    x = make("int8", [40, 8], 4, 2, 128, 16, seed=15)
    c = dev(x)
    call(c)
    for bad in (dict(scales=None), dict(scales=c["scales"][:-1]), dict(scales=c["scales"].half()), dict(scales=c["scales"][..., :1]),
                dict(k=c["k"].view(torch.uint8)), dict(v=c["v"].float().to(torch.float8_e4m3fn)), dict(k=c["k"].to(torch.bfloat16), v=c["v"].to(torch.bfloat16)),
                dict(scales=x["scales"]), dict(k=c["k"].transpose(1, 2))):
        with pytest.raises(ValueError):
            call({**c, **bad})
    with pytest.raises(CsaError) as e:
        call(c, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -1
    odd = torch.zeros(c["scales"].numel() + 2, device="cuda")[2:].view(c["scales"].shape)
    with pytest.raises(CsaError) as e:
        call({**c, "scales": odd})
    assert e.value.code == -3
