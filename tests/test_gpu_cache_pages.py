"""Page bookkeeping of the paged cache (reserve, free, fork, compact) and the
copies of pages, compared entry by entry with a host model."""
import random

import pytest
import torch

import continuous_softmax_attention_gb300 as csa
from continuous_softmax_attention_gb300 import CsaError, device_status
from paged_util import Books, pages_of

pytestmark = pytest.mark.gpu

INTS = dict(dtype=torch.int32, device="cuda")


class Device:
    """The state of a Books on the device, and the calls on it."""

    def __init__(self, m):
        self.m = m
        self.refs, self.table = torch.tensor(m.refs, **INTS), torch.tensor(m.table, **INTS).reshape(len(m.lens), m.M)
        self.lens = torch.tensor(m.lens, **INTS)

    @property
    def state(self):
        return self.refs, self.table, self.lens, self.m.S

    def equals(self):
        m = self.m
        assert self.refs.tolist() == m.refs
        assert self.lens.tolist() == m.lens
        assert self.table.tolist() == m.table

    def reserve(self, counts):
        return csa.cache_reserve(*self.state, torch.tensor(counts, **INTS)).item()

    def free(self, rows):
        csa.cache_free(*self.state, torch.tensor(rows, **INTS))

    def fork(self, p, c):
        return csa.cache_fork(*self.state, torch.tensor(p, **INTS), torch.tensor(c, **INTS))


def grown(B, P, S, M, counts):
    m = Books(B, P, S, M)
    d = Device(m)
    assert d.reserve(counts) == m.reserve(counts) == 0
    d.equals()
    return m, d


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("B,P,S,M", [(1, 5, 8, 4), (7, 40, 16, 8), (200, 3000, 16, 300), (40, 700, 8, 25), (1500, 9000, 24, 7), (33, 40000, 5, 1200)])
def test_a_long_run_of_everything(B, P, S, M, seed):
    r = random.Random(seed)
    m = Books(B, P, S, M)
    d = Device(m)
    for step in range(12):
        what = r.choice(["reserve", "reserve", "free", "fork", "compact"])
        if what == "reserve":
            most = r.choice([1, 3, S, 3 * S, M * S])
            counts = [min(r.randint(0, most), m.M * S - n) if r.random() < 0.8 else 0 for n in m.lens]
            want = m.reserve(counts)
            assert d.reserve(counts) == want
        elif what == "free":
            rows = [r.randrange(-1, B) for _ in range(r.randint(1, max(1, B // 2)))]
            m.free(rows)
            d.free(rows)
        elif what == "fork":
            empty = [b for b in range(B) if m.lens[b] == 0]
            kids = r.sample(empty, r.randint(0, len(empty)))
            if not kids:
                continue
            parents = [r.randrange(-1, B) for _ in kids]
            src, dst, short = d.fork(parents, kids)
            assert (src.tolist(), dst.tolist(), short.item()) == m.fork(parents, kids)
        else:
            src, dst, moved = csa.cache_compact(*d.state)
            ws, wd = m.compact()
            k = moved.item()
            pad = [-1] * (P // 2 - k)
            assert k == len(ws) and src.tolist() == ws + pad and dst.tolist() == wd + pad
        d.equals()
    assert device_status() == 0


def test_reserve_all_or_nothing():
    m, d = grown(3, 10, 16, 9, [30, 0, 17])
    assert d.reserve([16, 96, 16]) == m.reserve([16, 96, 16]) == 2  # 8 pages wanted, 6 free
    d.equals()
    assert d.reserve([0, 96, 0]) == 0 and m.reserve([0, 96, 0]) == 0  # exactly the rest
    d.equals()
    assert device_status() == 0
    for bad in ([0, 0, -1], [0, 49, 0], [2 ** 31 - 1, 0, 0]):
        assert d.reserve(bad) == -1
        assert device_status() == -1
        d.equals()


def test_free_refuses_and_repeats():
    m, d = grown(4, 12, 16, 4, [40, 16, 1, 0])
    d.free([0, 4])  # no row 4: nothing happens
    assert device_status() == -1
    d.equals()
    d.free([0, -2])
    assert device_status() == -1
    d.equals()
    d.free([1, -1, 1, 3, 1])
    m.free([1, -1, 1, 3, 1])
    d.equals()
    d.free([])
    assert device_status() == 0
    d.refs[m.table[0][1]] = 0  # a broken state: a held page that nobody holds
    d.table[0, 2] = 77
    d.free([0])
    assert device_status() == -1
    assert min(d.refs.tolist()) == 0 and d.lens[0] == 0


def test_fork_shares_and_refuses():
    m, d = grown(8, 20, 16, 5, [35, 32, 0, 7, 0, 0, 0, 0])
    for p, c in (([0, 1], [2, 2]), ([0], [1]), ([0], [8]), ([9], [2]), ([0, 0], [2, 0])):
        src, dst, short = d.fork(p, c)
        assert short.item() == -1 and src.tolist() == dst.tolist() == [-1] * len(p)
        assert device_status() == -1
        d.equals()
    p, c = [0, 0, -1, 1, 2, 3], [2, 4, 5, 6, 7, -1]  # twice the same parent, padding, a full last page, an empty parent
    src, dst, short = d.fork(p, c)
    assert (src.tolist(), dst.tolist(), short.item()) == m.fork(p, c)
    d.equals()
    m.free([0]), d.free([0])  # the pages live on with the children
    d.equals()
    assert max(m.refs) == 2
    m, d = grown(6, 30, 16, 300, [100, 0, 0, 0, 0, 0])
    p, c = [1, 0, 2, 4], [2, 1, 3, 5]  # parents that are children of the same call were empty: so are their children
    src, dst, short = d.fork(p, c)
    assert (src.tolist(), dst.tolist(), short.item()) == m.fork(p, c)
    assert m.lens == [100, 100, 0, 0, 0, 0]
    d.equals()
    m, d = grown(3, 3, 16, 2, [20, 3, 0])
    src, dst, short = d.fork([1], [2])  # no page left for the child's copy
    assert short.item() == 1 and src.tolist() == [-1] and m.fork([1], [2])[2] == 1
    d.equals()
    assert device_status() == 0


def test_many_forks_at_once():
    B, n = 5000, 4096
    m, d = grown(B, 30000, 8, 3, [1 + b % 24 for b in range(900)] + [0] * (B - 900))
    r = random.Random(1)
    p, c = [r.randrange(-1, 900) for _ in range(n)], r.sample(range(900, B), n)
    src, dst, short = d.fork(p, c)
    assert (src.tolist(), dst.tolist(), short.item()) == m.fork(p, c) and short.item() == 0
    d.equals()
    with pytest.raises(CsaError):
        d.fork([0] * (n + 1), [1] * (n + 1))


@pytest.mark.parametrize("dtype,shape", [(torch.bfloat16, (50, 2, 16, 128)), (torch.bfloat16, (3, 50, 4, 24, 64)),
                                         (torch.float32, (50, 1, 5, 7)), (torch.bfloat16, (2, 50, 1, 3, 5)),
                                         (torch.uint8, (50, 3, 8, 40)), (torch.bfloat16, (1, 50, 8, 256, 128))])
def test_copy_pages(dtype, shape):
    g = torch.Generator().manual_seed(len(shape))
    pool = lambda: torch.randint(0, 100, shape, generator=g).to(dtype).cuda()
    src, dst = [3, 7, 7, -1, 20, 49], [0, 1, 2, 30, -1, 48]
    for values in (pool(), None):
        k, v = pool(), values
        want = [t.clone() for t in (k, v) if t is not None]
        for t in want:
            for s, d in zip(src, dst):
                if s >= 0 and d >= 0:
                    t.select(-4, d).copy_(t.select(-4, s))
        csa.cache_copy_pages(k, v, torch.tensor(src, **INTS), torch.tensor(dst, **INTS))
        assert torch.equal(k, want[0]) and (v is None or torch.equal(v, want[1]))
    k0 = k.clone()
    csa.cache_copy_pages(k, None, torch.tensor([9, 10], **INTS), torch.tensor([11, 12], **INTS), count=torch.tensor([1], **INTS))
    k0.select(-4, 11).copy_(k0.select(-4, 9))
    assert torch.equal(k, k0)
    assert device_status() == 0
    csa.cache_copy_pages(k, None, torch.tensor([50, 1], **INTS), torch.tensor([1, 50], **INTS))
    assert device_status() == -1 and torch.equal(k, k0)


def test_refusals():
    m, d = grown(3, 10, 16, 4, [10, 0, 40])
    refs, table, lens, S = d.state
    one = torch.zeros(3, **INTS)
    for bad in (lambda: csa.cache_reserve(refs.long(), table, lens, S, one), lambda: csa.cache_reserve(refs, table.t(), lens, S, one),
                lambda: csa.cache_reserve(refs, table, lens, S, one[:2]), lambda: csa.cache_free(refs, table, lens.cpu(), S, one),
                lambda: csa.cache_free(refs, table, lens, S, one.float()), lambda: csa.cache_fork(refs, table, lens, S, one, one[:1]),
                lambda: csa.cache_compact(refs, table[0], lens, S), lambda: csa.cache_copy_pages(refs, None, one, one),
                lambda: csa.cache_reserve(refs, table, lens, S, one, stream=0)):
        with pytest.raises((ValueError, AttributeError)):
            bad()
    for bad in (lambda: csa.cache_reserve(refs, table, lens, 0, one),
                lambda: csa.cache_compact(refs, table, lens, -1)):
        with pytest.raises(CsaError) as e:
            bad()
        assert e.value.code == -1
    with pytest.raises(CsaError) as e:
        csa.cache_reserve(refs, table, lens, 2 ** 30, one)
    assert e.value.code == -2
    d.equals()


def test_a_server_step_by_step():
    """Prompts, forks, decode steps, a compaction and frees, with the attention of
    every step against the contiguous decode on the same tokens."""
    B, Hq, Hkv, d, S, P, M = 6, 8, 2, 128, 16, 64, 12
    g = torch.Generator().manual_seed(3)
    m = Books(B, P, S, M)
    dev = Device(m)
    plan = csa.RopeAxes(d, (16, 24, 24))
    kp, vp = torch.zeros(2, P, Hkv, S, d, dtype=torch.bfloat16, device="cuda").unbind()
    kc, vc = torch.zeros(2, B, Hkv, M * S, d, dtype=torch.bfloat16, device="cuda").unbind()  # contiguous, rotated keys

    def step(counts, T):
        assert dev.reserve(counts) == m.reserve(counts) == 0
        x = torch.randn(B, T, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
        q, k, v = (t.transpose(1, 2) for t in (x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]))
        place = torch.tensor([[n - c + t for t in range(T)] for n, c in zip(m.lens, counts)], **INTS)
        pos = torch.stack([place, place // 7, place % 7])
        qr, kr = csa.rope(q, k, pos, plan)
        qo = csa.cache_append(k, v, kp, vp, dev.table, dev.lens, counts=torch.tensor(counts, **INTS), rope=plan, positions=pos, q=q)
        assert torch.equal(qo, qr)
        for b, c in enumerate(counts):
            if c:
                kc[b, :, m.lens[b] - c:m.lens[b]], vc[b, :, m.lens[b] - c:m.lens[b]] = kr[b, :, :c], v[b, :, :c]
        last = torch.stack([qr[b, :, max(c, 1) - 1] for b, c in enumerate(counts)])
        o, lse = csa.decode_paged(last, kp, vp, dev.table, dev.lens, mode=csa.COPY_FIRST)
        rep = Hq // Hkv
        oc, lc = csa.decode(last, kc.repeat_interleave(rep, 1), vc.repeat_interleave(rep, 1), mode=csa.COPY_FIRST,
                            seqlens=dev.lens.clamp(min=1))
        for b, n in enumerate(m.lens):
            if n:  # two roundings to bf16 of nearly the same number
                assert ((o[b].float() - oc[b].float()).abs() <= 2.0 ** -7 * oc[b].float().abs() + 1e-4).all()
                assert (lse[b] - lc[b]).abs().max().item() <= 1e-5
            else:
                assert not o[b].any()

    def fork(p, c):
        src, dst, short = dev.fork(p, c)
        assert m.fork(p, c)[2] == short.item() == 0
        csa.cache_copy_pages(kp, vp, src, dst)
        for a, b in zip(p, c):
            kc[b], vc[b] = kc[a], vc[a]

    step([33, 16, 0, 0, 50, 0], 50)
    fork([0, 0, 1], [2, 3, 5])
    for _ in range(3):
        step([1, 1, 1, 1, 1, 1], 1)
    m.free([0, 4]), dev.free([0, 4])
    src, dst, moved = csa.cache_compact(*dev.state)
    csa.cache_copy_pages(kp, vp, src, dst, count=moved)
    m.compact()
    dev.equals()
    step([20, 1, 1, 1, 0, 5], 20)
    for _ in range(2):
        step([1, 1, 1, 1, 0, 1], 1)
    dev.equals()
    assert device_status() == 0


def test_a_captured_step():
    """reserve, append and decode of one token captured once and replayed."""
    B, Hq, Hkv, d, S, P, M = 4, 4, 2, 64, 8, 40, 6
    m, dev = grown(B, P, S, M, [7, 3, 0, 16])
    g = torch.Generator().manual_seed(5)
    plan = csa.RopeAxes(d, (32,))
    kp, vp = torch.randn(2, P, Hkv, S, d, generator=g).to(torch.bfloat16).cuda().unbind()
    x = torch.randn(B, Hq + 2 * Hkv, 1, d, generator=g).to(torch.bfloat16).cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    counts = torch.tensor([1, 1, 0, 1], **INTS)

    def step():
        short = csa.cache_reserve(*dev.state, counts)
        qo = csa.cache_append(k, v, kp, vp, dev.table, dev.lens, counts=counts, rope=plan, q=q)
        return (short,) + csa.decode_paged(qo[:, :, 0], kp, vp, dev.table, dev.lens)

    saved = [t.clone() for t in (dev.refs, dev.table, dev.lens, kp, vp)]
    eager = []
    for _ in range(5):
        eager.append([t.clone() for t in step()])
    for t, s in zip((dev.refs, dev.table, dev.lens, kp, vp), saved):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for want in eager:
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        m.reserve([1, 1, 0, 1])
        dev.equals()
    assert max(pages_of(n, S) for n in m.lens) == 3 and device_status() == 0


def test_pages_in_a_graph_and_on_a_given_stream():
    """free, fork and its copies, compaction and its moves captured once and replayed
    from other states, then the same calls on a stream of their own."""
    S, P, M, B = 8, 60, 6, 8
    g = torch.Generator().manual_seed(9)
    states = []
    for counts in ([30, 17, 8, 0, 0, 40, 5, 1], [9, 40, 0, 0, 0, 33, 48, 0], [3, 1, 7, 0, 0, 2, 0, 8]):
        m = Books(B, P, S, M)
        assert m.reserve(counts) == 0
        m.free([6])
        states.append(m)
    dev = Device(states[0])
    kp = torch.randn(2, P, 2, S, 64, generator=g).to(torch.bfloat16).cuda()
    rows, p, c = (torch.tensor(x, **INTS) for x in ([5, -1], [0, 1, 0], [3, 4, 6]))

    def step(**kw):
        csa.cache_free(*dev.state, rows, **kw)
        src, dst, short = csa.cache_fork(*dev.state, p, c, **kw)
        csa.cache_copy_pages(kp, None, src, dst, **kw)
        msrc, mdst, moved = csa.cache_compact(*dev.state, **kw)
        csa.cache_copy_pages(kp, None, msrc, mdst, count=moved, **kw)
        return short, moved

    def content(m, pages):  # what every sequence reads, whatever the pages are called
        return [pages[:, [m.table[b][j] for j in range(pages_of(n, S))]].clone() for b, n in enumerate(m.lens)]

    def load(m):
        for t, x in ((dev.refs, m.refs), (dev.table, m.table), (dev.lens, m.lens)):
            t.copy_(torch.tensor(x, **INTS).reshape(t.shape))
        dev.m = m

    load(states[0])
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        short, moved = step()
    side = torch.cuda.Stream()
    for run in ("graph", "stream"):
        for m0 in states:
            m = Books(B, P, S, M)
            m.refs, m.table, m.lens = list(m0.refs), [list(r) for r in m0.table], list(m0.lens)
            load(m)
            pages = kp.clone()
            m.free([5])
            assert m.fork([0, 1, 0], [3, 4, 6])[2] == 0
            before = content(m, pages)  # a copied page holds what its source held ...
            for child, parent in ((3, 0), (4, 1), (6, 0)):
                if m.lens[child] % S:
                    before[child][:, -1] = pages[:, m.table[parent][m.lens[parent] // S]]
            m.compact()
            torch.cuda.synchronize()
            if run == "graph":
                graph.replay()
            else:
                short, moved = step(stream=side)
            torch.cuda.synchronize()
            dev.equals()
            assert short.item() == 0
            assert all(torch.equal(x, y) for x, y in zip(content(m, kp), before))
    assert device_status() == 0


@pytest.mark.parametrize("M", [5, 3000])  # both forms of the rows' copy
def test_fork_of_a_broken_row(M):
    m, d = grown(3, 20, 16, M, [35, 32, 0])
    d.table[0, 1] = 20  # a shared page that the pool has not got
    src, dst, short = d.fork([0], [2])
    assert short.item() == 0 and device_status() == -1
    assert d.table[2].tolist()[:4] == [d.table[0, 0].item(), 20, dst.item(), -1]
    assert d.refs[d.table[0, 0]] == 2 and d.lens.tolist() == [35, 32, 35]
    m, d = grown(3, 20, 16, M, [35, 32, 0])
    d.table[0, 2] = 20  # the page that would be copied
    refs, table = d.refs.clone(), d.table.clone()
    src, dst, short = d.fork([0], [2])
    assert short.item() == -1 and device_status() == -1 and src.tolist() == dst.tolist() == [-1]
    assert torch.equal(d.refs, refs) and torch.equal(d.table, table) and d.lens.tolist() == [35, 32, 0]
