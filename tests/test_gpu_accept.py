"""The accepted branch of a draft kept (csa_cache_accept) and rows moved
(csa_cache_copy_rows), against the host's books."""
import numpy as np
import pytest
import torch

from continuous_softmax_attention_gb300 import CsaError, cache_accept, cache_copy_rows, cache_reserve, device_status
from draft_util import DraftBooks, path_of, random_pools, tree
from paged_util import pages_of

pytestmark = pytest.mark.gpu
INT = dict(dtype=torch.int32, device="cuda")


def books(lens, P, S, M, seed):
    """A host model and its state on the device: pages scattered over the pool."""
    m = DraftBooks(len(lens), P, S, M)
    order, at = np.random.default_rng(seed).permutation(P), 0
    for b, n in enumerate(lens):
        for j in range(pages_of(n, S)):
            m.table[b][j] = int(order[at])
            m.refs[order[at]] = 1
            at += 1
        m.lens[b] = n
    return m, torch.tensor(m.refs, **INT), torch.tensor(m.table, **INT), torch.tensor(m.lens, **INT)


def moved(pool, src, dst, S):
    """The pool after the rows of each group have moved, one group after the other."""
    out = pool.clone()
    for s, d in zip(src, dst):
        for i, j in zip(s, d):
            if i >= 0 and j >= 0:
                out[..., j // S, :, j % S, :] = pool[..., i // S, :, i % S, :]
    return out


@pytest.mark.parametrize("shape", ["chain", "star", "wide", "random"])
@pytest.mark.parametrize("T,S", [(1, 16), (5, 3), (16, 8), (33, 16), (64, 7), (64, 1)])
def test_against_the_host(shape, T, S):
    r = np.random.default_rng(T * S)
    B = 9
    counts = [int(r.integers(0, T + 1)) for _ in range(B)]
    counts[0] = T
    lens = [int(r.integers(0, 40)) + c for c in counts]
    lens[1] = counts[1]  # nothing before the draft
    parents = [tree(T, shape, r) for _ in range(B)]
    last = [int(r.integers(-1, c)) for c in counts]
    last[0] = T - 1
    m, refs, table, seq = books(lens, sum(pages_of(n, S) for n in lens) + 4, S, max(pages_of(n, S) for n in lens) + 1, T)
    kw = dict(counts=torch.tensor(counts, **INT))
    if shape != "chain":
        kw["parents"] = torch.tensor(parents, **INT)
    src, dst = cache_accept(refs, table, seq, S, torch.tensor(last, **INT), T, **kw)
    want_src, want_dst = m.accept(parents, counts, last, T)
    assert src.tolist() == want_src and dst.tolist() == want_dst
    assert refs.tolist() == m.refs and table.tolist() == m.table and seq.tolist() == m.lens
    assert device_status() == 0
    for kind in ("bf16", "int8"):
        k, v, scales = random_pools(m.P, 2, S, 24, kind, torch.Generator().manual_seed(1))
        u = [None if x is None else x.cuda() for x in (k, v, scales)]
        cache_copy_rows(u[0], u[1], src, dst, row_scales=u[2])
        for got, was in zip(u, (k, v, scales)):
            assert was is None or torch.equal(got.cpu(), moved(was, want_src, want_dst, S))


def test_without_counts_every_sequence_has_all():
    m, refs, table, seq = books([9, 4, 30], 20, 4, 9, 2)
    src, dst = cache_accept(refs, table, seq, 4, torch.tensor([1, -1, 3], **INT), 4)
    assert (src.tolist(), dst.tolist()) == m.accept([[-1, 0, 1, 2]] * 3, [4] * 3, [1, -1, 3], 4)
    assert seq.tolist() == m.lens == [7, 0, 30] and refs.tolist() == m.refs and table.tolist() == m.table
    assert (src == -1).all()  # a chain's kept tokens stay
    short = cache_reserve(refs, table, seq, 4, torch.tensor([5, 1, 2], **INT))  # the pages are free again
    assert short.item() == m.reserve([5, 1, 2]) == 0 and table.tolist() == m.table


def test_shared_pages_lose_one_holder():
    """A page that two sequences hold whole before the draft is not touched; one given back by both falls by two."""
    S = 4
    refs, table = torch.tensor([2, 1, 1, 2, 0], **INT), torch.tensor([[0, 1, 3], [0, 2, 3]], **INT)
    seq = torch.tensor([9, 10], **INT)
    src, dst = cache_accept(refs, table, seq, S, torch.tensor([0, 1], **INT), 5, counts=torch.tensor([3, 4], **INT))
    assert refs.tolist() == [2, 1, 1, 0, 0] and table.tolist() == [[0, 1, -1], [0, 2, -1]] and seq.tolist() == [7, 8]


def test_bad_sequences_stay_as_they_are():
    S, T = 4, 6
    lens = [10] * 8
    m, refs, table, seq = books(lens, 40, S, 4, 3)
    counts = [6, 7, -1, 6, 6, 6, 6, 6]
    last = [5, 0, 0, 6, -2, 5, 5, 5]
    parents = [[-1, 0, 1, 1, 1, 2] for _ in lens]
    parents[5][2] = 2      # itself
    parents[6][5] = -2
    table[7, 1] = 77       # rows 4..7 of it: node 2 at 6 among them
    before = [x.clone() for x in (refs, table, seq)]
    src, dst = cache_accept(refs, table, seq, S, torch.tensor(last, **INT), T, parents=torch.tensor(parents, **INT), counts=torch.tensor(counts, **INT))
    assert device_status() == -1 and device_status() == 0
    assert (src[1:] == -1).all() and (dst[1:] == -1).all() and torch.equal(seq[1:], before[2][1:]) and torch.equal(table[1:], before[1][1:])
    path = path_of(parents[0], 5)
    assert seq[0].item() == 4 + len(path) and (src[0] >= 0).sum().item() == sum(u != i for i, u in enumerate(path))
    assert (refs != before[0]).sum().item() == pages_of(10, S) - pages_of(4 + len(path), S)


def test_a_page_that_nobody_holds_is_passed_over():
    refs, table, seq = torch.tensor([1, 0, 1], **INT), torch.tensor([[0, 1, 9]], **INT), torch.tensor([9], **INT)
    cache_accept(refs, table, seq, 4, torch.tensor([-1], **INT), 8)
    assert refs.tolist() == [1, 0, 1] and seq.tolist() == [1] and table.tolist() == [[0, -1, -1]]
    assert device_status() == -1 and device_status() == 0


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float32), (256, torch.float32), (33, torch.int8), (6, torch.bfloat16), (1, torch.int8)])
@pytest.mark.parametrize("T", [1, 7, 64])
def test_rows_change_places(d, dtype, T):
    """A group's rows permuted among themselves, several layers; padding and rows out of range passed over."""
    g = torch.Generator().manual_seed(d)
    L, P, H, S, B = 3, 2 * T + 3, 2, 5, 4
    make = lambda *s: (torch.randn(*s, generator=g) * 50).to(dtype)  # noqa: E731
    k, v = make(L, P, H, S, d), make(L, P, H, S, d)
    order = torch.randperm(P * S, generator=g)[:B * T].view(B, T).int()
    src, dst = order, order[:, torch.randperm(T, generator=g)].contiguous()
    src, dst = src.clone(), dst.clone()
    if T > 2:
        src[0, 1], dst[1, 0], dst[2, 2] = -1, -5, P * S
    want_dst = torch.where(dst >= P * S, -1, dst)
    u, w = k.cuda(), v.cuda()
    cache_copy_rows(u, w, src.cuda(), dst.cuda())
    assert torch.equal(u.cpu(), moved(k, src.tolist(), want_dst.tolist(), S)) and torch.equal(w.cpu(), moved(v, src.tolist(), want_dst.tolist(), S))
    assert device_status() == (-1 if T > 2 else 0)
    u = k[0].contiguous().cuda()
    cache_copy_rows(u, None, src.cuda(), dst.cuda())
    assert torch.equal(u.cpu(), moved(k[0], src.tolist(), want_dst.tolist(), S))
    device_status()


@pytest.mark.parametrize("B,T,d,dtype", [(700, 3, 128, torch.bfloat16), (300, 20, 64, torch.float32), (130, 64, 96, torch.int8), (650, 9, 256, torch.float32)])
def test_many_groups(B, T, d, dtype):
    """More blocks than run at a time: a block has several planes, as many at once as fit, the last time fewer."""
    g = torch.Generator().manual_seed(B)
    L, H, S = 3, 5, 8
    P = B * T // S + 2
    k = (torch.randn(L, P, H, S, d, generator=g) * 50).to(dtype)
    order = torch.randperm(P * S, generator=g)[:B * T].view(B, T).int()
    dst = order[:, torch.randperm(T, generator=g)].contiguous()
    src = torch.where(torch.rand(B, T, generator=g) < 0.4, -1, order).int()
    u = k.cuda()
    cache_copy_rows(u, None, src.cuda(), dst.cuda())
    assert torch.equal(u.cpu(), moved(k, src.tolist(), dst.tolist(), S)) and device_status() == 0


def test_arguments_are_checked():
    m, refs, table, seq = books([5, 5], 6, 4, 2, 4)
    last = torch.tensor([0, 0], **INT)
    for kw in (dict(last=last[:1]), dict(last=last.long()), dict(last=last.cpu()), dict(T=-1), dict(parents=torch.zeros(2, 3, **INT)),
               dict(counts=torch.zeros(3, **INT))):
        a = dict(last=last, T=2) | kw
        with pytest.raises(ValueError):
            cache_accept(refs, table, seq, 4, a.pop("last"), a.pop("T"), **a)
    with pytest.raises(CsaError):
        cache_accept(refs, table, seq, 4, last, 65)
    k = torch.zeros(6, 1, 4, 8, device="cuda")
    one = torch.zeros(1, 1, **INT)
    for args, kw in (((k, k, one[0], one[0]), {}), ((k, k[:5], one, one), {}), ((k, k, one, one.long()), {}), ((k[:, :, :, :4], None, one, one), {}),
                     ((k, k, one, one), dict(row_scales=torch.zeros(6, 1, 4, 3, device="cuda"))), ((k[0], None, one, one), {})):
        with pytest.raises(ValueError):
            cache_copy_rows(*args, **kw)
    with pytest.raises(CsaError):
        cache_copy_rows(k, k, torch.zeros(1, 65, **INT), torch.zeros(1, 65, **INT))
    versions = [x._version for x in (refs, table, seq, k)]
    src, dst = cache_accept(refs, table, seq, 4, last, 2)
    cache_copy_rows(k, None, src, dst)
    assert all(x._version > n for x, n in zip((refs, table, seq, k), versions))
    for T in (0,):
        src, dst = cache_accept(refs, table, seq, 4, last, T)
        cache_copy_rows(k, None, src, dst)
        assert src.shape == (2, 0)


def test_in_a_graph():
    m, refs, table, seq = books([20, 11], 12, 4, 6, 5)
    parents, counts, last = [[-1, -1, 0, 1, 1, 3]] * 2, [6, 6], [5, 2]
    dev = [torch.tensor(x, **INT) for x in (parents, counts, last)]
    k, v, scales = (x.cuda() for x in random_pools(12, 2, 4, 16, "int8", torch.Generator().manual_seed(6)))
    state = [refs, table, seq, k, v, scales]
    begin = [x.clone() for x in state]
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        src, dst = cache_accept(refs, table, seq, 4, dev[2], 6, parents=dev[0], counts=dev[1])
        cache_copy_rows(k, v, src, dst, row_scales=scales)
    want_src, want_dst = m.accept(parents, counts, last, 6)
    for _ in range(2):
        for x, y in zip(state, begin):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert src.tolist() == want_src and seq.tolist() == m.lens and refs.tolist() == m.refs
        assert torch.equal(k.cpu(), moved(begin[3].cpu(), want_src, want_dst, 4)) and torch.equal(scales.cpu(), moved(begin[5].cpu(), want_src, want_dst, 4))
