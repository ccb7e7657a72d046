"""Attention of a tree of drafted tokens over pages (csa_decode_tree) against the CPU
oracle, which computes the last row of each node's own list of positions in 64 bits."""
import numpy as np
import pytest
import torch

import oracle
from continuous_softmax_attention_gb300 import (CsaError, decode_paged, decode_tree, decode_tree_workspace_bytes, device_status)
from draft_util import KINDS, bounds_tree, path_of, random_pools, tree, values
from paged_util import pages_of, rows_of, scattered

pytestmark = pytest.mark.gpu
KIND = pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
INT = dict(dtype=torch.int32, device="cuda")


def make(kind, past, counts, T, Hq, Hkv, d, S, seed, shape="random", spare=3, M=None):
    """past[b] tokens before counts[b] drafted ones."""
    g, r = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    lens = [n + c for n, c in zip(past, counts)]
    P = sum(pages_of(n, S) for n in lens) + spare
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    k, v, scales = random_pools(P, Hkv, S, d, kind, g)
    return dict(kind=kind, q=bf(len(lens), Hq, T, d), k=k, v=v, scales=scales, k0=bf(Hkv, d), v0=bf(Hkv, d), lens=lens, counts=list(counts),
                T=T, S=S, parents=[tree(T, shape, r) for _ in lens], table=scattered(lens, S, P, seed, M=M))


def dev(x):
    c = {n: t.cuda() for n, t in x.items() if torch.is_tensor(t)}
    return dict(c, table=torch.as_tensor(x["table"]).cuda(), lens=torch.tensor(x["lens"], **INT), counts=torch.tensor(x["counts"], **INT),
                parents=torch.tensor(x["parents"], **INT).view(len(x["lens"]), x["T"]))


def call(c, mode=0, scale=None, **kw):
    kw = dict(dict(counts=c["counts"], row_scales=c.get("scales")), **kw)
    return decode_tree(c["q"], c["k"], c["v"], c["table"], c["lens"], c["parents"], c["k0"], c["v0"], mode=mode, scale=scale, **kw)


def run(x, mode=0, scale=None, **kw):
    o, lse = call(dev(x), mode, scale, **kw)
    torch.cuda.synchronize()
    return o, lse


def check(x, o, lse, mode, scale=None, only=None, nodes=None, heads=None):
    B, Hq, T, d = x["q"].shape
    Hkv, S = x["k"].shape[1], x["S"]
    G, scale = Hq // Hkv, d ** -0.5 if scale is None else scale
    vk, vv = values(x["k"], x["v"], x["scales"])
    o, lse = o.double().cpu().numpy(), lse.cpu().numpy()
    for b in range(B) if only is None else only:
        n, c = x["lens"][b] - x["counts"][b], x["counts"][b]
        assert (o[b, :, c:] == 0).all() and np.isneginf(lse[b, :, c:]).all()
        k, v = (rows_of(t, x["table"][b], n + c, S) for t in (vk, vv))
        for t in range(c):
            if nodes is not None and t not in nodes:
                continue
            at = list(range(n)) + [n + u for u in path_of(x["parents"][b], t)]
            for h in range(Hq) if heads is None else heads:
                hk = h // G
                q = torch.zeros(1, 1, len(at), d, dtype=torch.float64)
                q[0, 0, -1] = x["q"][b, h, t].double()
                kk, vv_ = k[hk, at], v[hk, at]
                k0, v0 = x["k0"][hk:hk + 1].double(), x["v0"][hk:hk + 1].double()
                ro, rl = oracle.forward_rows(q, kk[None, None], vv_[None, None], [len(at) - 1], k0=k0, v0=v0, scale=scale, mode=mode)
                first = {0: (kk[:1] * 0, vv_[:1] * 0), 1: (kk[:1], vv_[:1]), 2: (k0, v0)}[mode]
                bo, bl = bounds_tree(x["kind"], G * T, x["q"][b, h, t].double(), torch.cat([first[0], kk]), torch.cat([first[1], vv_]), ro[0], rl[0], scale)
                err = np.abs(o[b, h, t] - ro[0])
                assert (err <= bo).all(), (b, h, t, n, float(err.max()), float((err / bo).max()))
                assert abs(lse[b, h, t] - rl[0]) <= bl, (b, h, t, n, float(lse[b, h, t]), float(rl[0]), bl)


PAST = [0, 1, 2, 7, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 130]


@KIND
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("T,G", [(5, 1), (3, 4), (16, 2), (9, 16)])
def test_pasts_around_every_edge(kind, mode, T, G):
    r = np.random.default_rng(T)
    counts = [int(r.integers(0, T + 1)) for _ in PAST]
    counts[0] = counts[1] = T
    x = make(kind, PAST, counts, T, G, 1, 64, 8, seed=T + mode)
    o, lse = run(x, mode)
    check(x, o, lse, mode, heads=None if G < 16 else (0, 7, 15))
    assert device_status() == 0


@KIND
@pytest.mark.parametrize("shape", ["chain", "star", "wide", "random"])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64])
def test_shapes_of_trees(kind, shape, T):
    x = make(kind, [40, 0, 200], [T, T, T - 1], T, 2, 1, 128, 16, seed=T, shape=shape)
    nodes = sorted({0, 1, T // 2, T - 2, T - 1} | set(range(30, 34)) & set(range(T)))
    for mode in (0, 1):
        o, lse = run(x, mode)
        check(x, o, lse, mode, nodes=nodes)


@KIND
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,T", [(1, 1, 1), (2, 2, 8), (8, 2, 4), (8, 2, 5), (6, 2, 11), (4, 1, 16), (4, 1, 31), (3, 1, 43), (33, 3, 12), (16, 2, 64), (8, 1, 17)])
def test_row_counts(kind, d, Hq, Hkv, T):
    """T times the heads of a group on every side of the blocks of rows."""
    x = make(kind, [5, 333, 0, 40, 1300], [T, T, 0, max(T - 1, 0), T], T, Hq, Hkv, d, 32, seed=Hq + T)
    o, lse = run(x, 2)
    check(x, o, lse, 2, nodes={0, T // 3, T - 2, T - 1}, heads=sorted({0, Hq // 2, Hq - 1}))


@KIND
@pytest.mark.parametrize("d,S,Hq,Hkv,T", [(128, 64, 8, 2, 16), (64, 256, 16, 2, 8), (256, 16, 4, 4, 3), (64, 8, 2, 1, 64)])
def test_long_and_ragged(kind, d, S, Hq, Hkv, T):
    x = make(kind, [20011, 1, 0, 4097, 300, 12000], [T, T, T, 1, 0, T - 1], T, Hq, Hkv, d, S, seed=d)
    o, lse = run(x, 0)
    check(x, o, lse, 0, nodes={0, T - 2, T - 1}, heads=(0, Hq - 1))


@KIND
def test_one_long_sequence_has_many_parts(kind):
    x = make(kind, [70003], [4], 4, 2, 1, 64, 64, seed=1)
    o, lse = run(x, 1)
    check(x, o, lse, 1)


@KIND
def test_many_short_sequences(kind):
    r = np.random.default_rng(5)
    past = [int(n) for n in r.integers(0, 90, 200)]
    counts = [int(n) for n in r.integers(0, 7, 200)]
    x = make(kind, past, counts, 6, 8, 4, 128, 16, seed=6)
    o, lse = run(x, 1)
    check(x, o, lse, 1, only=range(0, 200, 9), heads=(0, 5))


@KIND
@pytest.mark.parametrize("scale", [1.0, 4.0, -0.5, 0.0])
@pytest.mark.parametrize("T", [4, 24])
def test_logit_ranges(kind, scale, T):
    x = make(kind, [1, 30, 700], [T, T, T], T, 2, 1, 128, 16, seed=17)
    o, lse = run(x, 1, scale)
    check(x, o, lse, 1, scale, nodes={0, 2, T - 1})


@KIND
def test_a_chain_is_the_decode_steps_one_after_the_other(kind):
    T = 7
    x = make(kind, [100, 17, 0], [T, T, T], T, 4, 2, 128, 16, seed=8, shape="chain")
    c = dev(x)
    o, lse = call(c, 2)
    o2, l2 = decode_tree(c["q"], c["k"], c["v"], c["table"], c["lens"], None, c["k0"], c["v0"], row_scales=c.get("scales"), mode=2)
    assert torch.equal(o, o2) and torch.equal(lse, l2)  # no parents: a chain; no counts: all of them
    for t in range(T):
        a, la = decode_paged(c["q"][:, :, t].contiguous(), c["k"], c["v"], c["table"], c["lens"] - (T - 1 - t), c["k0"], c["v0"],
                             row_scales=c.get("scales"), mode=2)
        # two roundings to bf16 of nearly the same number, weights rounded to 2^-11 apart
        assert ((a.float() - o[:, :, t].float()).abs() <= 2.0 ** -7 * a.float().abs() + 2.0 ** -10 * x["v"].float().abs().max().item() * (1 if kind == "bf16" else x["scales"].max().item())).all()
        assert (la - lse[:, :, t]).abs().max().item() <= 1e-5


@KIND
@pytest.mark.parametrize("T", [6, 20])
def test_other_branches_and_rows_behind_may_hold_anything(kind, T):
    """Tokens that are not on a row's path, queries that are no node's, parents behind the counts and pages of nobody."""
    x = make(kind, [50, 3, 200], [T, T - 2, T], T, 2, 1, 128, 16, seed=9)
    for p in x["parents"]:
        p[:6] = [-1, 0, 0, 1, 2, 4]
        p[6:] = [t - 1 for t in range(6, T)]
    want, wl = run(x, 0)
    y = {n: t.clone() if torch.is_tensor(t) else t for n, t in x.items()}
    y["parents"] = [list(p) for p in x["parents"]]
    for b in range(3):  # node 3 hangs on 1: not above 2, 4, 5 and what follows
        at = x["lens"][b] - x["counts"][b] + 3
        page, slot = x["table"][b][at // 16], at % 16
        if kind == "bf16":
            y["k"][page, :, slot], y["v"][page, :, slot] = float("nan"), float("inf")
        else:
            y["scales"][page, :, slot] = float("nan")
            if kind == "e4m3":
                y["v"].view(torch.uint8)[page, :, slot] = 127
    y["q"][1, :, T - 2:] = float("nan")
    y["parents"][1][T - 2:] = [99, -7]
    held = {int(p) for b in range(3) for p in x["table"][b][:pages_of(x["lens"][b], 16)]}
    rest = [p for p in range(x["k"].shape[0]) if p not in held]
    (y["k"] if kind == "bf16" else y["scales"])[rest] = float("nan")
    o, lse = run(y, 0)
    clean = [t for t in range(T) if 3 not in path_of(x["parents"][0], t)]
    # the tokens of the others are read by the products of all: the same sums in another order
    assert ((o[:, :, clean].float() - want[:, :, clean].float()).abs() <= 2.0 ** -7 * want[:, :, clean].float().abs() + 1e-5).all()
    assert torch.equal(lse[:, :, clean], wl[:, :, clean]) and torch.isnan(o[:, :, 3].float()).all() and device_status() == 0


def test_infinite_values_on_the_path_pass_through():
    x = make("bf16", [50], [5], 5, 2, 1, 128, 16, seed=10, shape="star")
    x["v"][x["table"][0][51 // 16], 0, 51 % 16, 5] = float("inf")  # node 1
    x["v"][x["table"][0][1], 0, 3, 6] = float("-inf")              # before the draft
    o, _ = run(x, 0, 0.0)
    assert torch.isposinf(o[0, :, 1, 5]).all() and torch.isfinite(o[0, :, [0, 2, 3, 4], 5].float()).all() and torch.isneginf(o[0, :, :, 6]).all()
    assert torch.isfinite(o[..., 7:].float()).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T", [24, 64])
def test_infinite_values_with_many_rows(d, T):
    """Weights over bf16 pools are two numbers, neither of which may be 0 where the weight is not."""
    x = make("bf16", [300], [T], T, 2, 1, d, 16, seed=d)
    want, _ = run(x, 0, 0.5)
    for at, value in ((0, "inf"), (63, "-inf"), (64, "inf"), (200, "-inf"), (299, "inf")):
        y = dict(x, v=x["v"].clone())
        y["v"][x["table"][0][at // 16], 0, at % 16, 5] = float(value)
        o, _ = run(y, 0, 0.5)
        assert (o[..., 5].float() == float(value)).all(), at
        rest = [i for i in range(d) if i != 5]
        # The last row before the draft is also the tree's first position, whose values' infinities are summed one by one
        # with weights of 32 bits instead of two bf16 numbers (2^-16 of max |v|); and both sums are rounded, by half a step of
        # 2^-7 each.
        off = 2.0 ** -7 * want.float().abs() + 2.0 ** -16 * x["v"].float().abs().max().item() if at == 299 else 0.0
        assert ((o.float() - want.float()).abs() <= off)[..., rest].all(), at


@KIND
@pytest.mark.parametrize("d,B,Hkv,T,G", [(128, 40, 8, 64, 2), (256, 30, 8, 64, 2), (64, 60, 6, 31, 6), (256, 128, 8, 5, 3)])
def test_many_groups_of_rows(kind, d, B, Hkv, T, G):
    """More blocks than a few rounds of the GPU: a block then does several groups of rows.  Sequences of one tile
    (of 16 rows over bf16 pools with up to 16 rows per cached head, else of 32 and more) have the same parts in any batch,
    so the results are those of small batches bit for bit."""
    r = np.random.default_rng(d)
    past, counts = [int(n) for n in r.integers(0, 33, B)], [int(n) for n in r.integers(0, T + 1, B)]
    x = make(kind, past, counts, T, G * Hkv, Hkv, d, 8, seed=B)
    c = dev(x)
    o, lse = call(c, 1)
    for b in range(0, B, 10):
        part = slice(b, b + 2)
        few = dict(c, **{n: c[n][part].contiguous() for n in ("q", "table", "lens", "counts", "parents")})
        of, lf = call(few, 1)
        one = [n <= (16 if kind == "bf16" and G * T <= 16 else 32) for n in past[part]]
        assert torch.equal(o[part][one], of[one]) and torch.equal(lse[part][one], lf[one])
    check(x, o, lse, 1, only=(1, B - 1), nodes={0, T // 2, T - 1}, heads=(0, G * Hkv - 1))


def test_calls_of_other_sizes_at_once():
    """Kernels with other shares of an SM's tensor memory, registers and shared memory beside one another."""
    calls = []
    for kind, d, T, G in (("bf16", 128, 16, 4), ("bf16", 256, 64, 1), ("e4m3", 64, 31, 4), ("int8", 256, 20, 1), ("bf16", 64, 3, 2), ("e4m3", 128, 64, 2)):
        c = dev(make(kind, [900, 40, 0, 2000], [T] * 4, T, 2 * G, 2, d, 16, seed=d + T))
        o, lse = call(c)
        torch.cuda.synchronize()
        calls.append((c, o, lse, torch.cuda.Stream()))
    got = [[call(c, stream=s) for c, _, _, s in calls] for _ in range(8)]
    torch.cuda.synchronize()
    for some in got:
        for (c, o, lse, _), (a, b) in zip(calls, some):
            assert torch.equal(o, a) and torch.equal(lse, b)
    assert device_status() == 0


@KIND
@pytest.mark.parametrize("G", [1, 8])
def test_bad_lengths_pages_and_parents_are_reported(kind, G):
    T = 6
    x = make(kind, [100, 40, 60, 70, 30, 20, 33], [T] * 7, T, 2 * G, 2, 128, 16, seed=11)
    for p in x["parents"]:
        p[:] = [-1, 0, 1, 0, 3, 4]
    c = dev(x)
    call(c)
    assert device_status() == 0
    c["lens"][1] = c["table"].shape[1] * 16 + 1
    c["counts"][2] = T + 1
    c["lens"][3] = T - 1
    c["table"][4, 0] = -1                  # before the draft
    c["table"][5, (20 + T - 1) // 16] = 10 ** 6  # the draft's
    c["parents"][6, 3] = 3                 # its own parent: nodes 3, 4, 5
    o, lse = call(c)
    assert device_status() == -1 and device_status() == 0
    for b in range(1, 6):
        assert torch.isnan(o[b].float()).all() and torch.isnan(lse[b]).all(), b
    assert torch.isnan(o[6, :, 3:].float()).all() and torch.isnan(lse[6, :, 3:]).all() and torch.isfinite(o[6, :, :3].float()).all()
    heads = (0, 2 * G - 1)
    check(x, o, lse, 0, only=(0,), heads=heads)
    c["counts"][2], c["parents"][6, 3] = -1, -2
    o, _ = call(c)
    assert torch.isnan(o[2].float()).all() and torch.isnan(o[6, :, 3:].float()).all() and device_status() == -1


@KIND
@pytest.mark.parametrize("T,G", [(3, 1), (6, 8)])
def test_sequences_without_a_draft_are_passed_over(kind, T, G):
    x = make(kind, [500, 3000, 1, 40], [T, 0, 0, T - 1], T, 2 * G, 2, 128, 16, seed=15)
    x["table"][1, :], x["table"][2, :] = -1, 10 ** 6  # their pages are not looked at
    o, lse = run(x, 1)
    check(x, o, lse, 1, heads=(0, 2 * G - 1), only=(0, 3))
    assert (o[1:3] == 0).all() and torch.isneginf(lse[1:3]).all() and device_status() == 0
    x.update(counts=[0] * 4, lens=[500, 3000, 0, 40])
    o, lse = run(x, 1)
    assert (o == 0).all() and torch.isneginf(lse).all() and device_status() == 0


@KIND
@pytest.mark.parametrize("T", [3, 20])
def test_repeats_bit_for_bit_on_stale_workspaces(kind, T):
    x = make(kind, [3000, 17, 0, 900], [T] * 4, T, 8, 2, 128, 32, seed=12)
    o, lse = run(x, 0)
    n = decode_tree_workspace_bytes(4, 8, 2, T, 128)
    for fill in (255, 0, 127):
        o2, l2 = run(x, 0, workspace=torch.full((n,), fill, dtype=torch.uint8, device="cuda"))
        assert torch.equal(o, o2) and torch.equal(lse, l2)


@KIND
@pytest.mark.parametrize("T", [4, 24])
def test_streams_and_a_graph_with_other_trees(kind, T):
    x = make(kind, [500, 300, 20], [T, 2, T], T, 4, 2, 64, 16, seed=14)
    c = dev(x)
    o, lse = call(c)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for i in range(9):
        got.append(call(c, stream=streams[i % 3]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) and torch.equal(lse, b) for a, b in got)
    graph = torch.cuda.CUDAGraph()
    ws = torch.empty(decode_tree_workspace_bytes(3, 4, 2, T, 64), dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(graph):
        o, lse = call(c, workspace=ws)
    for i, (lens, counts) in enumerate((([500 + T, 302, 20 + T], [T, 2, T]), ([T, 299, 0], [T, 0, 0]), ([480, 1, 17], [1, 1, 2]))):
        x.update(lens=lens, counts=counts, parents=[tree(T, "random", np.random.default_rng(i)) for _ in lens])
        c["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        c["counts"].copy_(torch.tensor(counts, dtype=torch.int32))
        c["parents"].copy_(torch.tensor(x["parents"], dtype=torch.int32))
        ws.fill_(i + 1)
        graph.replay()
        torch.cuda.synchronize()
        check(x, o, lse, 0, nodes={0, 1, T - 1}, heads=(0, 3))


def test_no_pool_and_empty_calls():
    e = torch.zeros(0, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(2, 2, **INT)
    o, lse = decode_tree(q, e, e, table, torch.zeros(2, **INT), counts=torch.zeros(2, **INT))
    assert not o.any() and torch.isneginf(lse).all() and device_status() == 0
    o, lse = decode_tree(q, e, e, table, torch.tensor([0, 5], **INT), counts=torch.tensor([0, 2], **INT))
    assert not o[0].any() and torch.isnan(o[1].float()).all() and device_status() == -1
    for shape in ((0, 4, 3, 64), (2, 4, 0, 64)):
        o, lse = decode_tree(torch.ones(*shape, dtype=torch.bfloat16, device="cuda"), e, e, table[:shape[0]], torch.zeros(shape[0], **INT))
        assert o.shape == shape and lse.shape == shape[:3]


def test_pages_beyond_32_bits():
    P, Hkv, S, d, T = 40000, 4, 64, 256, 5
    x = make("bf16", [300, 1000], [T, T], T, 8, Hkv, d, S, seed=31)
    far = {p: (P - 1 - p if p % 2 else p) for p in range(x["k"].shape[0])}
    k, v = (torch.zeros(P, Hkv, S, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for p, f in far.items():
        k[f], v[f] = x["k"][p].cuda(), x["v"][p].cuda()
    c = dev(x)
    c.update(k=k, v=v, table=torch.as_tensor([[far.get(int(e), -1) for e in row] for row in x["table"]], dtype=torch.int32).cuda())
    o, lse = call(c)
    check(x, o, lse, 0, nodes={0, 4}, heads=(0, 7))


def test_refusals():
    x = make("int8", [40, 8], [3, 3], 3, 4, 2, 128, 16, seed=15)
    c = dev(x)
    call(c)
    for bad in (dict(parents=c["parents"][:, :2]), dict(parents=c["parents"].long()), dict(counts=c["counts"][:1]), dict(scales=None),
                dict(q=c["q"].float()), dict(q=c["q"][0]), dict(q=c["q"].transpose(1, 2)), dict(table=c["table"].long()),
                dict(k=c["k"].float(), v=c["v"].float(), scales=None)):
        with pytest.raises(ValueError):
            call({**c, **bad})
    with pytest.raises(ValueError):
        decode_tree(c["q"], c["k"], c["v"], c["table"], c["lens"], row_scales=c["scales"], mode=2)
    for kw, over, code in ((dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), {}, -1), (dict(scale=float("nan")), {}, -1),
                           ({}, dict(q=torch.zeros(2, 4, 65, 128, dtype=torch.bfloat16, device="cuda"), parents=torch.zeros(2, 65, **INT)), -2),
                           ({}, dict(q=c["q"][:, :3].contiguous()), -1)):
        with pytest.raises(CsaError) as e:
            call({**c, **over}, **kw)
        assert e.value.code == code
    with pytest.raises(CsaError):
        decode_tree_workspace_bytes(1, 8, 2, 65, 128)
