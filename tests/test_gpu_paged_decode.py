"""Decode step over a paged cache (csa_decode_paged) against the CPU oracle,
which computes row n - 1 of eq. (8) in 64 bits from the same bf16 values."""
import numpy as np
import pytest
import torch

import oracle
from continuous_softmax_attention_gb300 import (CsaError, decode, decode_paged,
                                                decode_paged_workspace_bytes, device_status)
from paged_util import decode_bounds, pages_of, rows_of, scattered

pytestmark = pytest.mark.gpu


FORMS = pytest.mark.parametrize("wide", [False, True], ids=["one kernel", "parts joined"])


def make(lens, Hq, Hkv, d, S, seed, spare=3, wide=False):
    """wide: a table for sequences of 40000 tokens, with which even short ones are
    cut over all workers and their parts joined by a second kernel."""
    g = torch.Generator().manual_seed(seed)
    P = sum(pages_of(n, S) for n in lens) + spare
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    x = dict(q=bf(len(lens), Hq, d), k=bf(P, Hkv, S, d), v=bf(P, Hkv, S, d), k0=bf(Hkv, d), v0=bf(Hkv, d))
    x["table"] = scattered(lens, S, P, seed, M=pages_of(40000, S) if wide else None)
    x["lens"] = list(lens)
    return x


def run(x, mode=0, scale=None, **kw):
    c = {n: t.cuda() for n, t in x.items() if torch.is_tensor(t)}
    o, lse = decode_paged(c["q"], c["k"], c["v"], torch.as_tensor(x["table"]).cuda(),
                          torch.tensor(x["lens"], dtype=torch.int32).cuda(), c["k0"], c["v0"], mode=mode, scale=scale, **kw)
    torch.cuda.synchronize()
    return o, lse


def check(x, o, lse, S, mode, scale, only=None):
    """Every (sequence, head), or the listed sequences, against the oracle."""
    B, Hq, d = x["q"].shape
    Hkv = x["k"].shape[1]
    o, lse = o.float().cpu().numpy(), lse.cpu().numpy()
    for b in range(B) if only is None else only:
        n = x["lens"][b]
        if n == 0:
            assert (o[b] == 0).all() and np.isneginf(lse[b]).all()
            continue
        k, v = (rows_of(x[t], x["table"][b], n, S) for t in ("k", "v"))
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            q = torch.zeros(1, 1, n, d)
            q[0, 0, n - 1] = x["q"][b, h].float()
            ro, rl = oracle.forward_rows(q, k[None, hk:hk + 1].float(), v[None, hk:hk + 1].float(), [n - 1],
                                         k0=x["k0"][hk:hk + 1].float(), v0=x["v0"][hk:hk + 1].float(), scale=scale, mode=mode)
            first = {0: (k[hk, :1] * 0, v[hk, :1] * 0), 1: (k[hk, :1], v[hk, :1]),
                     2: (x["k0"][hk:hk + 1], x["v0"][hk:hk + 1])}[mode]
            bo, bl = decode_bounds(x["q"][b, h].float(), torch.cat([first[0], k[hk]]).float(),
                                   torch.cat([first[1], v[hk]]).float(), ro[0], rl[0], scale)
            err = np.abs(o[b, h] - ro[0])
            assert (err <= bo).all(), (b, h, n, float(err.max()), float((err / bo).max()))
            assert abs(lse[b, h] - rl[0]) <= bl, (b, h, n, float(lse[b, h]), float(rl[0]), bl)


EDGES = [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 0, 127, 128, 129, 200]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("S", [8, 16, 24, 64])
@FORMS
def test_lengths_around_every_edge(d, mode, S, wide):
    x = make(EDGES, 2, 1, d, S, seed=d + S + mode, wide=wide)
    o, lse = run(x, mode)
    check(x, o, lse, S, mode, d ** -0.5)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (3, 1), (8, 2), (10, 2), (16, 1), (9, 1), (17, 1), (40, 2), (33, 11)])
@FORMS
def test_head_groups(Hq, Hkv, wide):
    x = make([5, 333, 0, 40, 1], Hq, Hkv, 128, 32, seed=Hq, wide=wide)
    o, lse = run(x, 2)
    check(x, o, lse, 32, 2, 128 ** -0.5)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.125, 1.0, 4.0, -0.5, 0.0])
@FORMS
def test_logit_ranges(d, scale, wide):
    # scale 4 gives steps between neighbouring logits of order 100
    x = make([1, 2, 30, 300, 700], 4, 2, d, 16, seed=17, wide=wide)
    o, lse = run(x, 1, scale)
    check(x, o, lse, 16, 1, scale)


@FORMS
def test_rising_and_falling_logits(wide):
    # one key direction with growing, falling and peaked weights: the running maximum moves late or never
    n, d = 500, 128
    x = make([n, n, n], 1, 1, d, 16, seed=3, wide=wide)
    u = torch.randn(d, generator=torch.Generator().manual_seed(1))
    ramp = torch.linspace(-30, 30, n)
    shapes = [ramp, ramp.flip(0), torch.where(torch.arange(n) == 377, torch.tensor(60.0), -ramp.abs())]
    x["q"][:] = u.to(torch.bfloat16)
    for b, s in enumerate(shapes):
        for i in range(n):
            x["k"][x["table"][b, i // 16], 0, i % 16] = (s[i] * u / u.norm() ** 2 * d ** 0.5).to(torch.bfloat16)
    o, lse = run(x, 0)
    check(x, o, lse, 16, 0, d ** -0.5)


@pytest.mark.parametrize("d,S,Hq,Hkv", [(128, 64, 8, 2), (64, 256, 16, 2), (256, 16, 4, 4), (64, 8, 2, 1)])
def test_long_and_ragged(d, S, Hq, Hkv):
    lens = [20011, 1, 0, 4097, 300, 12000]
    x = make(lens, Hq, Hkv, d, S, seed=d)
    o, lse = run(x, 0)
    check(x, o, lse, S, 0, d ** -0.5)


def test_many_short_sequences():
    lens = [int(n) for n in np.random.default_rng(5).integers(0, 90, 300)]
    x = make(lens, 8, 4, 128, 16, seed=6)
    o, lse = run(x, 1)
    check(x, o, lse, 16, 1, 128 ** -0.5, only=range(0, 300, 7))


@FORMS
def test_matches_the_contiguous_decode(wide):
    B, H, T, d, S = 3, 4, 700, 128, 16
    lens = [700, 333, 1]
    x = make(lens, H, H, d, S, seed=8, wide=wide)
    kc, vc = torch.zeros(2, B, H, T, d, dtype=torch.bfloat16).unbind()
    for b, n in enumerate(lens):
        kc[b, :, :n], vc[b, :, :n] = rows_of(x["k"], x["table"][b], n, S), rows_of(x["v"], x["table"][b], n, S)
    for mode in (0, 1, 2):
        o, lse = run(x, mode)
        oc, lc = decode(x["q"].cuda(), kc.cuda(), vc.cuda(), x["k0"].cuda(), x["v0"].cuda(), mode=mode,
                        seqlens=torch.tensor(lens, dtype=torch.int32).cuda())
        # two roundings to bf16 of nearly the same number
        assert ((o.float() - oc.float()).abs() <= 2.0 ** -7 * oc.float().abs() + 1e-4).all()
        assert (lse - lc).abs().max().item() <= 1e-5


@FORMS
def test_pages_hold_anything_behind_the_last_token(wide):
    # rows behind a sequence's end, and pages of nobody, are NaN or infinite
    lens, S, d = [1, 17, 100, 129, 40], 16, 128
    x = make(lens, 4, 2, d, S, seed=9, wide=wide)
    want, wl = run(x, 0)
    held = set()
    for b, n in enumerate(lens):
        ids = x["table"][b, :pages_of(n, S)]
        held.update(ids.tolist())
        for t in ("k", "v"):
            if n % S:
                x[t][ids[-1], :, n % S:] = float("nan") if t == "k" else float("inf")
    rest = [p for p in range(x["k"].shape[0]) if p not in held]
    x["k"][rest], x["v"][rest] = float("nan"), float("nan")
    o, lse = run(x, 0)
    assert torch.equal(o, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("Hq", [1, 8, 16])
@pytest.mark.parametrize("scale", [0.0, 0.1])
@FORMS
def test_infinite_values_in_the_cache_pass_through(Hq, scale, wide):
    # scale 0: the weights are exact in bf16
    x = make([50, 2000], Hq, 1, 128, 16, seed=10, wide=wide)
    for b, n in ((0, 1), (1, 100)):
        x["v"][x["table"][b, n], 0, 3, 5], x["v"][x["table"][b, n], 0, 4, 6] = float("inf"), float("-inf")
    o, _ = run(x, 0, scale)
    assert torch.isposinf(o[:, :, 5]).all() and torch.isneginf(o[:, :, 6]).all()
    assert torch.isfinite(o[:, :, 7:].float()).all()


@FORMS
def test_sequences_that_share_pages(wide):
    x = make([200, 75, 200], 4, 2, 64, 16, seed=30, wide=wide)
    x["table"][1, :5] = x["table"][0, :5]
    x["table"][2] = x["table"][0]
    o, lse = run(x, 2)
    check(x, o, lse, 16, 2, 64 ** -0.5)


def test_no_pool():
    e = torch.zeros(0, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    o, lse = decode_paged(q, e, e, table, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert not o.any() and torch.isneginf(lse).all() and device_status() == 0
    o, lse = decode_paged(q, e, e, table, torch.tensor([0, 5, 40], dtype=torch.int32, device="cuda"))
    assert not o[0].any() and torch.isnan(o[1:].float()).all() and device_status() == -1
    table.zero_()
    o, lse = decode_paged(q, e, e, table, torch.tensor([0, 5, 40], dtype=torch.int32, device="cuda"))
    assert torch.isnan(o[1:].float()).all() and device_status() == -1


def test_pages_beyond_32_bits():
    # pools of 2.3e9 elements (4.7 GB); the sequences' pages lie at both ends
    P, Hkv, S, d = 72000, 4, 64, 128
    lens = [300, 1000, 64]
    x = make(lens, 8, Hkv, d, S, seed=31)
    far = {p: (P - 1 - p if p % 2 else p) for p in range(x["k"].shape[0])}
    k, v = (torch.empty(P, Hkv, S, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for p, f in far.items():
        k[f], v[f] = x["k"][p].cuda(), x["v"][p].cuda()
    table = torch.as_tensor([[far.get(int(e), -1) for e in row] for row in x["table"]], dtype=torch.int32).cuda()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    o, lse = decode_paged(x["q"].cuda(), k, v, table, n)
    check(x, o, lse, S, 0, d ** -0.5)
    # the same pages by the other calls: rows written at the far end, and pages copied there
    from continuous_softmax_attention_gb300 import cache_append, cache_copy_pages

    new = torch.randn(3, Hkv, 1, d, device="cuda").to(torch.bfloat16)
    cache_append(new, new, k, v, table, n)
    for b, m in enumerate(lens):
        assert torch.equal(k[table[b, (m - 1) // S], :, (m - 1) % S], new[b, :, 0])
    cache_copy_pages(k, v, torch.tensor([0], dtype=torch.int32).cuda(), torch.tensor([P - 2], dtype=torch.int32).cuda())
    assert torch.equal(k[P - 2], k[0]) and torch.equal(v[P - 2], v[0])
    assert device_status() == 0


@FORMS
def test_bad_lengths_and_pages_are_reported(wide):
    S, d = 16, 128
    x = make([100, 40, 60, 70, 0], 4, 2, d, S, seed=11, wide=wide)
    run(x, 0)
    assert device_status() == 0
    P, M = x["k"].shape[0], x["table"].shape[1]
    x["lens"][1] = M * S + 1
    x["lens"][4] = -3
    x["table"][2, 1] = P  # one page too far, in the middle of a sequence
    o, lse = run(x, 0)
    assert device_status() == -1 and device_status() == 0
    for b in (1, 2, 4):
        assert torch.isnan(o[b].float()).all() and torch.isnan(lse[b]).all()
    # the others are right; their last bits may differ, as the parts are cut by all lengths
    check(x, o, lse, S, 0, d ** -0.5, only=(0, 3))
    x["table"][2, 1] = -1
    o, _ = run(x, 0)
    assert device_status() == -1 and torch.isnan(o[2].float()).all()


@FORMS
def test_repeats_bit_for_bit_on_stale_workspaces(wide):
    lens = [3000, 17, 0, 900, 5000]
    x = make(lens, 8, 2, 128, 32, seed=12, wide=wide)
    o, lse = run(x, 0)
    n = decode_paged_workspace_bytes(5, 8, 2, 128)
    for fill in (255, 0, 127):
        o2, l2 = run(x, 0, workspace=torch.full((max(n, 16),), fill, dtype=torch.uint8, device="cuda"))
        assert torch.equal(o, o2) and torch.equal(lse, l2)


@FORMS
def test_two_streams_and_a_given_stream(wide):
    x = make([2000, 900, 50], 8, 2, 128, 16, seed=13, wide=wide)
    o, lse = run(x, 0)
    c = {n: t.cuda() for n, t in x.items() if torch.is_tensor(t)}
    table, lens = torch.as_tensor(x["table"]).cuda(), torch.tensor(x["lens"], dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for i in range(30):
        got.append(decode_paged(c["q"], c["k"], c["v"], table, lens, stream=streams[i % 3]))
    torch.cuda.synchronize()
    for oo, ll in got:
        assert torch.equal(o, oo) and torch.equal(lse, ll)


@FORMS
def test_captured_and_replayed_with_other_lengths(wide):
    x = make([500, 300, 20], 4, 2, 64, 16, seed=14, wide=wide)
    c = {n: t.cuda() for n, t in x.items() if torch.is_tensor(t)}
    table, lens = torch.as_tensor(x["table"]).cuda(), torch.tensor(x["lens"], dtype=torch.int32).cuda()
    decode_paged(c["q"], c["k"], c["v"], table, lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = decode_paged(c["q"], c["k"], c["v"], table, lens)
    for now in ([500, 300, 20], [1, 299, 0], [480, 1, 17]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        x["lens"] = now
        check(x, o, lse, 16, 0, 64 ** -0.5)


@FORMS
def test_two_graphs_on_one_workspace(wide):
    a, b = make([700, 30, 0], 8, 2, 128, 16, seed=40, wide=wide), make([5, 900], 8, 2, 128, 32, seed=41, wide=wide)
    n = max(decode_paged_workspace_bytes(3, 8, 2, 128), decode_paged_workspace_bytes(2, 8, 2, 128))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    held, graphs = [], []
    for x in (a, b):
        c = {t: x[t].cuda() for t in ("q", "k", "v")}
        table, lens = torch.as_tensor(x["table"]).cuda(), torch.tensor(x["lens"], dtype=torch.int32).cuda()
        want = decode_paged(c["q"], c["k"], c["v"], table, lens, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = decode_paged(c["q"], c["k"], c["v"], table, lens, workspace=ws)
        held.append((c, table, lens, want, got))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0, 0):  # one after the other on one stream
        for t in held[i][4]:
            t.zero_()
        graphs[i].replay()
        graphs[1 - i].replay()
        torch.cuda.synchronize()
        for _, _, _, want, got in held:
            assert all(torch.equal(w, t) for w, t in zip(want, got))


def test_refusals():
    x = make([40, 8], 4, 2, 128, 16, seed=15)
    c = {n: t.cuda() for n, t in x.items() if torch.is_tensor(t)}
    table, lens = torch.as_tensor(x["table"]).cuda(), torch.tensor(x["lens"], dtype=torch.int32).cuda()
    ok = dict(q=c["q"], k=c["k"], v=c["v"], table=table, lens=lens)

    def call(kw=None, **over):
        a = {**ok, **over}
        return decode_paged(a["q"], a["k"], a["v"], a["table"], a["lens"], **(kw or {}))

    call()
    for bad in (dict(q=c["q"].float()), dict(k=c["k"].half()), dict(v=c["v"][:-1]), dict(table=table.long()),
                dict(lens=lens[:1]), dict(k=c["k"].transpose(1, 2)), dict(q=c["q"][0]), dict(q=x["q"])):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError):
        call(dict(mode=2))
    for kw, over, code in ((dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), {}, -1),
                           (dict(scale=float("nan")), {}, -1), (dict(mode=3), {}, -1),
                           ({}, dict(q=c["q"][:, :3].contiguous()), -1),
                           ({}, dict(k=c["k"][:, :, :12].contiguous(), v=c["v"][:, :, :12].contiguous()), -2),
                           ({}, dict(k=c["k"][..., :96].contiguous(), v=c["v"][..., :96].contiguous(),
                                     q=c["q"][..., :96].contiguous()), -2)):
        with pytest.raises(CsaError) as e:
            call(kw, **over)
        assert e.value.code == code
    o, lse = call(q=c["q"][:0], table=table[:0], lens=lens[:0])
    assert o.shape == (0, 4, 128) and lse.shape == (0, 4)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (10, 2), (16, 1), (17, 1), (9, 3)])
@FORMS
def test_head_groups_of_other_widths(d, Hq, Hkv, wide):
    x = make([5, 333, 0, 40, 1, 1500], Hq, Hkv, d, 24, seed=Hq + d, wide=wide)
    for mode in (0, 1, 2):
        o, lse = run(x, mode)
        check(x, o, lse, 24, mode, d ** -0.5)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("Hq", [2, 24])
@FORMS
def test_garbage_infinities_and_repeats_of_other_widths(d, Hq, wide):
    lens, S = [1, 17, 100, 0, 129, 2040], 8
    x = make(lens, Hq, 2, d, S, seed=d + Hq, wide=wide)
    want, wl = run(x, 0)
    held = set()
    for b, n in enumerate(lens):
        ids = x["table"][b, :pages_of(n, S)]
        held.update(ids.tolist())
        if n % S:
            x["k"][ids[-1], :, n % S:], x["v"][ids[-1], :, n % S:] = float("nan"), float("inf")
    rest = [p for p in range(x["k"].shape[0]) if p not in held]
    x["k"][rest], x["v"][rest] = float("nan"), float("nan")
    need = decode_paged_workspace_bytes(len(lens), Hq, 2, d)
    for fill in (255, 0, 127):
        o, lse = run(x, 0, workspace=torch.full((max(need, 16),), fill, dtype=torch.uint8, device="cuda"))
        assert torch.equal(o, want) and torch.equal(lse, wl)
    # an infinite value in either half of the columns; a page out of range
    x["v"][x["table"][2, 3], :, 2, 5], x["v"][x["table"][5, 9], :, 1, d - 3] = float("inf"), float("-inf")
    x["table"][4, 1] = x["k"].shape[0]
    o, lse = run(x, 0, 0.0)
    assert torch.isposinf(o[2, :, 5]).all() and torch.isneginf(o[5, :, d - 3]).all()
    assert torch.isfinite(o[2, :, 6:].float()).all() and torch.isfinite(o[5, :, :d - 3].float()).all()
    assert torch.isnan(o[4].float()).all() and torch.isnan(lse[4]).all() and device_status() == -1
