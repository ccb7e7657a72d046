"""The calls of a server with drafted tokens together: room reserved, drafts appended at
their depths, their attention, the accepted branch kept and moved, the next token
decoded.  Against a cache that only ever saw the accepted tokens, and in a graph."""
import numpy as np
import pytest
import torch

import continuous_softmax_attention_gb300 as csa
from draft_util import KINDS, path_of, tree

pytestmark = pytest.mark.gpu
INT = dict(dtype=torch.int32, device="cuda")
B, HQ, HKV, D, S, M, P, T, L = 3, 4, 2, 64, 8, 12, 40, 9, 2


class Cache:
    """L layers of pools over one table."""

    def __init__(self, kind):
        shape = (L, P, HKV, S, D)
        self.kind = kind
        if kind == "bf16":
            self.k, self.v, self.scales = torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), None
        else:
            self.k, self.v = (torch.zeros(shape, device="cuda").to(KINDS[kind]) for _ in range(2))
            self.scales = torch.zeros(*shape[:-1], 2, device="cuda")
        self.refs, self.table, self.lens = torch.zeros(P, **INT), torch.full((B, M), -1, **INT), torch.zeros(B, **INT)
        self.plan = csa.RopeAxes(D, (D // 2,))

    def layer(self, i):
        return (self.k[i], self.v[i]), (dict(row_scales=self.scales[i]) if self.scales is not None else {})

    def reserve(self, counts):
        return csa.cache_reserve(self.refs, self.table, self.lens, S, counts)

    def append(self, i, k, v, q, counts, positions):
        pools, kw = self.layer(i)
        return csa.cache_append(k, v, *pools, self.table, self.lens, counts=counts, rope=self.plan, positions=positions, q=q, **kw)

    def rows(self, i, t):
        pools, kw = self.layer(i)
        return csa.cache_read(*pools, self.table, self.lens, t, **kw)


def step(c, x, parents, counts, last, depth):
    """One verification: returns the shortfall and the outputs of both layers' trees."""
    short = c.reserve(counts)
    positions = (c.lens - counts)[:, None] + depth
    outs = []
    for i in range(L):
        q = c.append(i, x[i, 1], x[i, 2], x[i, 0], counts, positions)
        pools, kw = c.layer(i)
        outs.append(csa.decode_tree(q, *pools, c.table, c.lens, parents, counts=counts, **kw)[0])
    src, dst = csa.cache_accept(c.refs, c.table, c.lens, S, last, T, parents=parents, counts=counts)
    csa.cache_copy_rows(c.k, c.v, src, dst, row_scales=c.scales)
    return short, outs


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_a_server_with_drafts(kind):
    r, g = np.random.default_rng(0), torch.Generator().manual_seed(0)
    drafted, plain = Cache(kind), Cache(kind)
    held = [0] * B
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    for round_ in range(6):
        counts = [int(r.integers(1, T + 1)) for _ in range(B)]
        parents = [tree(T, ("random", "wide", "chain")[round_ % 3], r) for _ in range(B)]
        last = [int(r.integers(-1, c)) for c in counts]
        paths = [path_of(p, t) for p, t in zip(parents, last)]
        depth = torch.tensor([[len(path_of(p, t)) - 1 for t in range(T)] for p in parents], **INT)
        x = bf(L, 3, B, HQ, T, D)
        qkv = [[x[i, 0], x[i, 1, :, :HKV], x[i, 2, :, :HKV]] for i in range(L)]
        class X:  # x[i, j] of one layer
            def __getitem__(self, ij):
                return qkv[ij[0]][ij[1]]
        short, outs = step(drafted, X(), torch.tensor(parents, **INT), torch.tensor(counts, **INT), torch.tensor(last, **INT), depth)
        # the plain cache: the accepted tokens alone, one path after the other, row by row
        kept = [len(p) for p in paths]
        n = torch.tensor(kept, **INT)
        assert short.item() == 0 and plain.reserve(n).item() == 0
        at = torch.tensor([p + [0] * (T - len(p)) for p in paths], device="cuda")[:, None, :, None].expand(B, HQ, T, D)
        for i in range(L):
            q, k, v = (t.gather(2, at[:, :t.shape[1]]) for t in qkv[i])
            plain.append(i, k, v, q, n, None)
        held = [a + b for a, b in zip(held, kept)]
        assert drafted.lens.tolist() == plain.lens.tolist() == held
        for i in range(L):
            for a, b in zip(drafted.rows(i, max(held) + 1), plain.rows(i, max(held) + 1)):
                assert torch.equal(a, b)
        assert (drafted.refs > 0).sum().item() == sum(-(-h // S) for h in held)
        assert all(torch.isfinite(o.float()).all() for o in outs)
        # the row of the last accepted node is the plain cache's decode step
        for i in range(L):
            pools, kw = plain.layer(i)
            for b in range(B):
                if not kept[b]:
                    continue
                q1 = csa.rope(qkv[i][0][b:b + 1, :, last[b]:last[b] + 1].contiguous(), None, torch.tensor([[[held[b] - 1]]], **INT), plain.plan)[0]
                o, _ = csa.decode_paged(q1[:, :, 0], *pools, plain.table[b:b + 1], plain.lens[b:b + 1], **kw)
                # two roundings to bf16 of nearly the same number; weights to 2^-8, 2^-11 apart
                big = max(t.float().abs().max().item() for t in plain.rows(i, max(held))[1:])
                assert ((outs[i][b, :, last[b]].float() - o[0].float()).abs() <= 2.0 ** -7 * o[0].float().abs() + 2.0 ** -8 * big).all()
    assert csa.device_status() == 0


def test_the_step_in_a_graph():
    r, g = np.random.default_rng(1), torch.Generator().manual_seed(1)
    caches = [Cache("int8"), Cache("int8")]
    x = torch.randn(L, 3, B, HQ, T, D, generator=g).to(torch.bfloat16).cuda()

    class X:
        def __getitem__(self, ij):
            return x[ij[0], ij[1]] if ij[1] == 0 else x[ij[0], ij[1], :, :HKV]

    parents, depth = torch.zeros(B, T, **INT), torch.zeros(B, T, **INT)
    counts, last = torch.zeros(B, **INT), torch.zeros(B, **INT)

    def draw():
        p = [tree(T, "random", r) for _ in range(B)]
        parents.copy_(torch.tensor(p, dtype=torch.int32))
        depth.copy_(torch.tensor([[len(path_of(q, t)) - 1 for t in range(T)] for q in p], dtype=torch.int32))
        n = [int(r.integers(1, T + 1)) for _ in range(B)]
        counts.copy_(torch.tensor(n, dtype=torch.int32))
        last.copy_(torch.tensor([int(r.integers(-1, c)) for c in n], dtype=torch.int32))

    draw()
    step(caches[0], X(), parents, counts, last, depth)  # also warms up
    step(caches[1], X(), parents, counts, last, depth)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        short, outs = step(caches[1], X(), parents, counts, last, depth)
    for _ in range(4):
        draw()
        x.copy_(torch.randn(x.shape, generator=g))
        want_short, want = step(caches[0], X(), parents, counts, last, depth)
        graph.replay()
        torch.cuda.synchronize()
        assert short.item() == want_short.item() == 0 and all(torch.equal(a, b) for a, b in zip(outs, want))
        assert torch.equal(caches[0].table, caches[1].table) and torch.equal(caches[0].lens, caches[1].lens) and torch.equal(caches[0].refs, caches[1].refs)
    for i in range(L):
        assert all(torch.equal(a, b) for a, b in zip(caches[0].rows(i, 60), caches[1].rows(i, 60)))
    assert csa.device_status() == 0
