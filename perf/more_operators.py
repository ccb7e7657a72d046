"""Serving operators for drafted tokens and 8-bit caches: the cases they are timed and compared on.

Five operators over the paged key-value cache of continuous softmax attention, and what stands between them:

* ``decode`` - one decode step over a cache held in 8 bits (e4m3 or int8, one scale per cached row and head);
* ``tree``   - attention of a tree of drafted tokens over the cache that already holds their rows: each drafted token
               sees the tokens before the draft and its own ancestors, over bf16 and 8-bit pools;
* ``fill``   - new tokens' rows quantised as they are written into their pages (keys rotated on the way, queries
               rotated beside) and read back as the values that the cache now stands for;
* ``read``   - rows of the cache read back in order, in 16 bits;
* ``accept`` - after the verification: the accepted branch's rows moved together, pages that fall empty given back.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the calls of this repository's
package.  A case is a dict of plain values; lengths, trees and accepted nodes are drawn from the case's own
``lens_seed`` so that the work does not depend on the seed of the contents.
"""
import math
import random

import torch

own = False

ZERO, COPY_FIRST, GIVEN = 0, 1, 2
LAWS = ("uniform", "log", "full")
TREES = ("chain", "random", "wide")


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user, a short chat, every head with its own keys, 8-bit cache: the latency of a single small step
        dict(name="decode_one_short", op="decode", kind="e4m3", B=1, Hq=32, Hkv=32, d=128, S=16, lo=1, hi=333, law="full",
             empty=0, mode=ZERO, lens_seed=1),
        # a server's batch under continuous batching: ragged lengths over three decades, four query heads on a cached
        # head, a few places of the batch unused
        dict(name="decode_ragged_grouped", op="decode", kind="int8", B=64, Hq=32, Hkv=8, d=128, S=16, lo=1, hi=8192,
             law="log", empty=5, mode=COPY_FIRST, lens_seed=2),
        # the benchmark's decode workload (16 sequences of 4096 to 8192 tokens, 32 heads) in 8 bits
        dict(name="decode_headline", op="decode", kind="e4m3", B=16, Hq=32, Hkv=32, d=128, S=64, lo=4096, hi=8192,
             law="uniform", empty=0, mode=ZERO, lens_seed=6),
        # one user, five drafted tokens in a row behind a short chat, bf16 cache: latency
        dict(name="tree_one_short", op="tree", kind="bf16", B=1, Hq=32, Hkv=8, d=128, S=16, lo=1, hi=333, law="full",
             T=5, empty=0, tree="chain", full=True, mode=ZERO, lens_seed=3),
        # a server's batch verifying trees of 16 drafted tokens, four query heads on a cached head, bf16 cache
        dict(name="tree_server", op="tree", kind="bf16", B=16, Hq=32, Hkv=8, d=128, S=64, lo=4096, hi=8192, law="uniform",
             T=16, empty=0, tree="random", full=False, mode=COPY_FIRST, lens_seed=4),
        # trees of 64 tokens behind long documents in an 8-bit cache of narrow heads, eight queries each, given sinks
        dict(name="tree_long_d64", op="tree", kind="e4m3", B=2, Hq=16, Hkv=2, d=64, S=32, lo=60001, hi=65000, law="uniform",
             T=64, empty=0, tree="wide", full=True, mode=GIVEN, lens_seed=5),
        # the new token of each sequence of a batch, quantised into its page and read back: latency
        dict(name="fill_step", op="fill", kind="e4m3", B=64, T=1, Hq=32, Hkv=8, d=128, S=16, sections="16,24,24",
             dtype="bf16", past=1000, lens_seed=8),
        # ragged prompts of up to 2048 tokens filled into the cache behind what is there, and read back
        dict(name="fill_prompt", op="fill", kind="int8", B=8, T=2048, Hq=32, Hkv=8, d=128, S=64, sections="16,24,24",
             dtype="bf16", past=777, lens_seed=9),
        # the last tokens of a batch of short caches, for a caller's own window attention
        dict(name="read_windows", op="read", kind="e4m3", B=32, T=128, Hkv=8, d=128, S=16, lo=1, hi=1000, law="uniform",
             lens_seed=10),
        # whole caches handed over to a contiguous attention or another server
        dict(name="read_caches", op="read", kind="int8", B=16, T=8192, Hkv=8, d=128, S=64, lo=4096, hi=8192, law="uniform",
             lens_seed=11),
        # a chat server after verifying chains of 8 drafted tokens: the tail given up, nothing to move
        dict(name="accept_chains", op="accept", kind="e4m3", B=64, T=8, Hkv=8, d=128, S=16, L=1, lo=1, hi=2000,
             law="uniform", tree="chain", lens_seed=12),
        # the same after trees of 64, eight layers of bf16 pools at once
        dict(name="accept_trees", op="accept", kind="bf16", B=64, T=64, Hkv=8, d=128, S=16, L=8, lo=1, hi=300,
             law="uniform", tree="random", lens_seed=13),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sections(rng, d):
    half = d // 2
    total = half if rng.random() < 0.5 else rng.randint(max(1, half // 3), half)
    axes = min(rng.choice([1, 2, 3, 4]), total)
    cuts = sorted(rng.sample(range(1, total), axes - 1)) if axes > 1 else []
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def _pairs(case):
    """Rotated pairs of each axis, from the case's text."""
    return [int(n) for n in case["sections"].split(",")]


def draw(rng):
    op = rng.choice(["decode", "decode", "tree", "tree", "tree", "fill", "read", "accept"])
    ls = rng.randint(0, 1 << 30)
    eight = rng.choice(["e4m3", "int8"])
    if op in ("decode", "tree"):
        d = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 3, 4, 8, 8])
        G = min(rng.choice([1, 1, 2, 3, 4, 4, 5, 7, 8, 16]), 64 // Hkv)
        T = 1 if op == "decode" else rng.choice([1, 2, 3, 5, 8, 16, 16, 31, 64, rng.randint(1, 64)])
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 131072)
        hi = max(1, min(hi, 12 * 8192 * 8 * 128 // (B * Hkv * d), 2 ** 33 // (B * Hkv * G * T * d)))
        law = rng.choice(LAWS)
        case = dict(op=op, kind=eight, B=B, Hq=G * Hkv, Hkv=Hkv, d=d, S=rng.choice([8, 16, 24, 32, 48, 64, 128, 256]),
                    lo=rng.randint(1, hi) if law == "uniform" else 1, hi=hi, law=law, empty=rng.randint(0, B // 3),
                    mode=rng.choice([ZERO, COPY_FIRST, GIVEN]), lens_seed=ls)
        if op == "decode":
            return case
        return dict(case, kind=rng.choice(["bf16", "bf16", eight]), T=T, tree=rng.choice(TREES), full=rng.random() < 0.5)
    d = rng.choice([64, 128, 128, 256, 96, 80])
    Hkv = rng.choice([1, 2, 4, 8])
    B = _log_int(rng, 1, 64)
    S = rng.choice([8, 16, 24, 64, 128])
    if op == "fill":
        T = rng.choice([1, 1, 2, _log_int(rng, 1, 2048)])
        T = max(1, min(T, 8 * 2048 * 8 * 128 // (B * Hkv * d)))
        return dict(op=op, kind=eight, B=B, T=T, Hq=Hkv * rng.choice([1, 2, 4]), Hkv=Hkv, d=d, S=S, sections=_sections(rng, d),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), past=_log_int(rng, 1, 1000), lens_seed=ls)
    if op == "read":
        hi = _log_int(rng, 1, 8192)
        hi = max(1, min(hi, 16 * 8192 * 8 * 128 // (2 * B * Hkv * d)))
        return dict(op=op, kind=rng.choice(["bf16", eight, eight]), B=B, T=rng.randint(1, hi), Hkv=Hkv, d=d, S=S,
                    lo=rng.randint(1, hi), hi=hi, law=rng.choice(["uniform", "full"]), lens_seed=ls)
    return dict(op=op, kind=rng.choice(["bf16", eight]), B=B, T=rng.randint(1, 64), Hkv=Hkv, d=d, S=S, L=rng.choice([1, 2, 3]),
                lo=1, hi=_log_int(rng, 1, 300), law=rng.choice(LAWS), tree=rng.choice(TREES), lens_seed=ls)


def _lens(case):
    """Tokens that each sequence holds before the drafted or new ones: over [lo, hi] (or its logarithm, or all hi)."""
    r = random.Random(case["lens_seed"])
    lo, hi, law, n = case["lo"], case["hi"], case["law"], case["B"]
    lens = [hi if law == "full" else r.randint(lo, hi) if law == "uniform" else _log_int(r, lo, hi) for _ in range(n)]
    for i in r.sample(range(n), min(case.get("empty", 0), n)):
        lens[i] = 0
    return lens


def _trees(case):
    """The parent of each drafted token [B][T] (-1: it follows the cache) and how many of each sequence's count."""
    r, B, T = random.Random(case["lens_seed"] + 1), case["B"], case["T"]
    parents = []
    for _ in range(B):
        if case["tree"] == "chain":
            parents.append(list(range(-1, T - 1)))
        elif case["tree"] == "random":  # each token continues one of the last few, a few begin anew
            parents.append([-1 if t == 0 or r.random() < 0.1 else r.randint(max(0, t - 6), t - 1) for t in range(T)])
        else:  # every token has about four continuations
            parents.append([-1 if t == 0 else (t - 1) // 4 for t in range(T)])
    full = case.get("full", case["op"] == "accept")
    return parents, [T if full else r.randint(0, T) for _ in range(B)]


def _last(case):
    """The last accepted node of each sequence, -1 where the draft failed at once."""
    r, counts = random.Random(case["lens_seed"] + 2), _trees(case)[1]
    return [r.randint(-1, c - 1) for c in counts]


def _path(parents, t):
    """The nodes from a root down to t."""
    path = []
    while t >= 0:
        path.append(t)
        t = parents[t]
    return path[::-1]


def _pages(n, S):
    return -(-n // S)


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _tables(lens, S, P, g, M=None):
    """A block table [B, M] over scattered pages of a pool of P, -1 behind each sequence's own."""
    M = max([_pages(n, S) for n in lens] + [1]) if M is None else M
    need = torch.tensor([_pages(n, S) for n in lens], device="cuda")
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    at = (torch.cumsum(need, 0) - need)[:, None] + torch.arange(M, device="cuda")
    used = torch.arange(M, device="cuda") < need[:, None]
    return torch.where(used, order[at.clamp(max=P - 1)], torch.full_like(at, -1, dtype=torch.int32))


def _rows(g, *shape):
    """Rows as a projection leaves them: most columns alike, a few larger, rows of different lengths."""
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
    x[..., :: max(1, shape[-1] // 3)] *= 3
    return x.mul_(torch.exp2(0.5 * torch.randn(*shape[:-1], 1, generator=g, device="cuda")))


def _quantise(x, kind):
    """Codes and scales of rows x [..., d].  e4m3: the scale is the smallest power of two by which the largest magnitude
    is at most 448; int8: the largest magnitude / 127, the codes the integers nearest to x * (127 / that magnitude),
    which is formed in 64 bits since 32 would round it onto a tie.  Rows below 2^-100 are zeros."""
    most = x.abs().amax(-1, keepdim=True)
    none = most < 2.0 ** -100
    most = most.masked_fill(none, 1.0)
    if kind == "e4m3":
        m, e = torch.frexp(most)
        s = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).int())
        codes = (x / s).masked_fill(none, 0).to(torch.float8_e4m3fn)
    else:
        s = most / 127
        codes = torch.round(x.double() * (127 / most).double()).masked_fill(none, 0).to(torch.int8)
    return codes, s.masked_fill(none, 0)


def _pools(case, shape, g):
    """k_pages, v_pages of `shape` + [Hkv, S, d], and the rows' scales [..., Hkv, S, 2] of 8-bit ones."""
    shape = (*shape, case["Hkv"], case["S"], case["d"])
    if case["kind"] == "bf16":
        return dict(k_pages=_rows(g, *shape).to(torch.bfloat16), v_pages=_rows(g, *shape).to(torch.bfloat16), row_scales=None)
    k, ks = _quantise(_rows(g, *shape), case["kind"])
    v, vs = _quantise(_rows(g, *shape), case["kind"])
    return dict(k_pages=k, v_pages=v, row_scales=torch.cat([ks, vs], -1).contiguous())


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_decode(case, seed):
    g = _gen(seed)
    B, Hq, Hkv, d, S, T = (case.get(k, 1) for k in ("B", "Hq", "Hkv", "d", "S", "T"))
    tree = case["op"] == "tree"
    lens = _lens(case)
    parents, counts = _trees(case) if tree else (None, [0] * B)
    lens = [n + c for n, c in zip(lens, counts)]
    P = sum(_pages(n, S) for n in lens) + 7
    bf = dict(generator=g, device="cuda", dtype=torch.bfloat16)
    state = dict(_pools(case, (P,), g), q=torch.randn(B, Hq, T, d, **bf) if tree else torch.randn(B, Hq, d, **bf),
                 k0=torch.randn(Hkv, d, **bf), v0=torch.randn(Hkv, d, **bf), table=_tables(lens, S, P, g), seqlens=_ints(lens))
    if tree:
        state.update(parents=_ints(parents), counts=_ints(counts))
    if own:
        import continuous_softmax_attention_gb300 as csa

        size = csa.decode_tree_workspace_bytes(B, Hq, Hkv, T, d) if tree else csa.decode_paged_workspace_bytes(B, Hq, Hkv, d)
        state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return state


def _fill_lens(case):
    r = random.Random(case["lens_seed"])
    T = case["T"]
    counts = [T if T == 1 else r.randint(0, T) for _ in range(case["B"])]
    return [r.randint(0, case["past"]) + c for c in counts], counts


def _prepare_fill(case, seed):
    g = _gen(seed)
    B, T, Hq, Hkv, d, S = (case[k] for k in ("B", "T", "Hq", "Hkv", "d", "S"))
    lens, counts = _fill_lens(case)
    P = sum(_pages(n, S) for n in lens) + 5
    x = _rows(g, B, T, Hq + 2 * Hkv, d).to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    n, c = _ints(lens), _ints(counts)
    t = (n - c)[None, :, None] + torch.arange(T, device="cuda")
    state = dict(_pools(case, (P,), g), q=x[:, :, :Hq].transpose(1, 2), k=x[:, :, Hq:Hq + Hkv].transpose(1, 2),
                 v=x[:, :, Hq + Hkv:].transpose(1, 2), table=_tables(lens, S, P, g), seqlens=n, counts=c, starts=n - c,
                 positions=torch.cat([t, t // 29, t % 29, t % 7][:len(_pairs(case))]).to(torch.int32).contiguous())
    if own:
        import continuous_softmax_attention_gb300 as csa

        state["rope"] = csa.RopeAxes(d, _pairs(case))
    return state


def _prepare_read(case, seed):
    g = _gen(seed)
    lens, S = _lens(case), case["S"]
    P = sum(_pages(n, S) for n in lens) + 3
    return dict(_pools(case, (P,), g), table=_tables(lens, S, P, g), seqlens=_ints(lens),
                starts=_ints([max(0, n - case["T"]) for n in lens]))


def _prepare_accept(case, seed):
    g = _gen(seed)
    B, S, T = case["B"], case["S"], case["T"]
    parents, counts = _trees(case)
    lens = [n + c for n, c in zip(_lens(case), counts)]
    P = sum(_pages(n, S) for n in lens) + 9
    table = _tables(lens, S, P, g)
    refs = torch.bincount(table[table >= 0].to(torch.int64), minlength=P)
    # refs, table and seqlens as views of one buffer, and that buffer as it was: a pass begins from there
    meta = torch.cat([refs.to(torch.int32), table.reshape(-1), _ints(lens)])
    n = table.numel()
    return dict(_pools(case, (case["L"], P), g), meta=meta, meta0=meta.clone(), refs=meta[:P], table=meta[P:P + n].view(table.shape),
                seqlens=meta[P + n:], parents=_ints(parents), counts=_ints(counts), last=_ints(_last(case)), S=S)


def prepare(case, seed):
    state = dict(decode=_prepare_decode, tree=_prepare_decode, fill=_prepare_fill, read=_prepare_read,
                 accept=_prepare_accept)[case["op"]](case, seed)
    return dict(state, case=case)


# ------------------------------------------------------------------------------------- plain forms
def _shares(a, b, m):
    """What the interval between neighbouring logits a and b gives the key at a and the key at b: with x = b - a and
    phi2(x) = (e^x - 1 - x)/x^2, e^{a-m} phi2(x) and e^{b-m} phi2(-x)."""
    x, pa, pb = b - a, torch.exp(a - m), torch.exp(b - m)
    even = 0.5 + x * x * (1 / 24 + x * x * (1 / 720 + x * x * (1 / 40320 + x * x / 3628800)))
    odd = x * (1 / 6 + x * x * (1 / 120 + x * x * (1 / 5040 + x * x * (1 / 362880 + x * x / 39916800))))
    near, y = x.abs() < 1, torch.where(x == 0, torch.ones_like(x), x)
    return (torch.where(near, pa * (even + odd), ((pb - pa) / y - pa) / y),
            torch.where(near, pb * (even - odd), (pb - (pb - pa) / y) / y))


def _values(s):
    """The rows of every sequence in order, [B, Hkv, M * S, d] each, as 32-bit values."""
    B, M = s["table"].shape
    at = s["table"].clamp(min=0).long()
    k, v = s["k_pages"][at].float(), s["v_pages"][at].float()
    if s["row_scales"] is not None:
        scales = s["row_scales"][at]
        k, v = k * scales[..., :1], v * scales[..., 1:]
    Hkv, S, d = k.shape[2:]
    return [x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * S, d) for x in (k, v)]


def _ancestors(parents, there):
    """[B, T, T]: whether node u is t or one of its ancestors; parents of what is not there count for nothing."""
    T = parents.shape[1]
    step = (parents[:, :, None] == torch.arange(T, device="cuda")) & there[:, :, None]
    reach = torch.linalg.matrix_power(step.float() + torch.eye(T, device="cuda"), T)
    return (reach > 0) & there[:, :, None] & there[:, None, :]


def _plain_attention(s):
    """Rows t = 0..T-1 of query heads over the tokens before the draft (decode: all held tokens, T = 1, no draft)."""
    c = s["case"]
    tree = c["op"] == "tree"
    B, Hq, Hkv, d, T = (c.get(k, 1) for k in ("B", "Hq", "Hkv", "d", "T"))
    G, n = Hq // Hkv, s["seqlens"] - s["counts"] if tree else s["seqlens"]
    k, v = _values(s)
    N = k.shape[2]
    place = torch.arange(N, device="cuda")
    held = (place < s["seqlens"][:, None])[:, None, :, None]
    k, v = k.masked_fill(~held, 0), v.masked_fill(~held, 0)
    q = s["q"].float().reshape(B, Hkv, G * T, d) * d ** -0.5
    if c["mode"] == GIVEN:
        k0, v0 = (x.float()[None, :, None].expand(B, Hkv, 1, d) for x in (s["k0"], s["v0"]))
    else:
        k0, v0 = (x[:, :, :1] * (1 if c["mode"] == COPY_FIRST else 0) for x in (k, v))
    a = torch.cat([q @ k0.transpose(2, 3), q @ k.transpose(2, 3)], 3)  # positions 0 (the sink) to N
    there = (torch.arange(N + 1, device="cuda") <= n[:, None])[:, None, None]
    m = a.masked_fill(~there, -math.inf).amax(3, keepdim=True)
    if tree:
        # drafted node u is row n + u of the cache
        u = torch.arange(T, device="cuda")
        drafted = u < s["counts"][:, None]
        at = (n[:, None] + u).clamp(max=N - 1).long()[:, None, :, None].expand(B, Hkv, T, d)
        kn, vn = k.gather(2, at), v.gather(2, at)
        parents = s["parents"].long()
        seen = _ancestors(parents, drafted)[:, None, None].expand(B, Hkv, G, T, T).reshape(B, Hkv, G * T, T)
        an = q @ kn.transpose(2, 3)  # [B, Hkv, G * T, T]
        before = a.gather(3, n.long()[:, None, None, None].expand(B, Hkv, G * T, 1))  # the last position before the draft
        if c["mode"] == COPY_FIRST:  # no token before the draft: each row's sink is a copy of its own first token
            root = (seen & (parents < 0)[:, None, None]).float()
            alone = (n == 0)[:, None, None, None]
            before = torch.where(alone, (an * root).sum(3, keepdim=True), before)
            m = torch.where(alone, before, m)
        m = torch.maximum(m, an.masked_fill(~seen, -math.inf).amax(3, keepdim=True))
        up = parents.clamp(min=0)[:, None, None].expand(B, Hkv, G * T, T)
        ap = torch.where((parents >= 0)[:, None, None], an.gather(3, up), before)
        nl, nr = (x.masked_fill(~seen, 0) for x in _shares(ap, an, m))
    left, right = _shares(a[..., :-1], a[..., 1:], m)
    gap = there[..., 1:]  # the interval up to a position exists if the position does
    w = torch.zeros_like(a)
    w[..., :-1] += left.masked_fill(~gap, 0)
    w[..., 1:] += right.masked_fill(~gap, 0)
    none = (n == 0)[:, None, None]
    if tree:
        first = (parents < 0)[:, None, None]
        joint = (nl * first).sum(3, keepdim=True)  # what the last position before the draft gets
        w.scatter_add_(3, n.long()[:, None, None, None].expand(B, Hkv, G * T, 1), joint)
        wn = nr + torch.zeros_like(nl).scatter_add_(3, up, nl * ~first)
        l = w.sum(3) + wn.sum(3)
        o = w[..., :1] @ v0 + w[..., 1:] @ v + wn @ vn
        if c["mode"] == COPY_FIRST:
            o = torch.where(alone, joint * (root @ vn) + wn @ vn, o)
        none = ~drafted[:, None, None].expand(B, Hkv, G, T).reshape(B, Hkv, G * T)
    else:
        l = w.sum(3)
        o = w[..., :1] @ v0 + w[..., 1:] @ v
    o = (o / l[..., None]).masked_fill(none[..., None], 0)
    lse = (m[..., 0] + torch.log(l)).masked_fill(none, -math.inf)
    shape = (B, Hq, T) if tree else (B, Hq)
    return dict(o=o.reshape(*shape, d).to(torch.bfloat16), lse=lse.reshape(shape))


def _plain_rotate(x, positions, case):
    """x [B, H, T, d] with its pairs turned by position * 10000^(-i / pairs), in 32 bits; angles in 64 bits."""
    axis = torch.repeat_interleave(torch.arange(len(_pairs(case)), device="cuda"), torch.tensor(_pairs(case), device="cuda"))
    n = axis.numel()
    f = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / n)
    angle = (positions.double()[axis].permute(1, 2, 0) * f)[:, None]  # [B, 1, T, pairs]
    cos, sin, y = torch.cos(angle).float(), torch.sin(angle).float(), x.float()
    u, w = y[..., :n], y[..., n:2 * n]
    return torch.cat([u * cos - w * sin, u * sin + w * cos, y[..., 2 * n:]], -1)


def _plain_read(s, T):
    """Rows starts .. starts + T - 1 of every sequence, [B, Hkv, T, d] each; 0 behind a sequence's end."""
    t = s["starts"][:, None] + torch.arange(T, device="cuda")
    seen = t < s["seqlens"][:, None]
    S, M = s["case"]["S"], s["table"].shape[1]
    page = s["table"].gather(1, (t // S).clamp(max=M - 1).long()).clamp(min=0).long()
    row = (t % S).long()
    k, v = s["k_pages"][page, :, row].float(), s["v_pages"][page, :, row].float()  # [B, T, Hkv, d]
    if s["row_scales"] is not None:
        scales = s["row_scales"][page, :, row]
        k, v = k * scales[..., :1], v * scales[..., 1:]
    return [x.masked_fill(~seen[..., None, None], 0).transpose(1, 2).to(torch.bfloat16).contiguous() for x in (k, v)]


def _plain_fill(s):
    c = s["case"]
    T, S = c["T"], c["S"]
    t = torch.arange(T, device="cuda")
    b, i = torch.nonzero(t < s["counts"][:, None], as_tuple=True)
    at = ((s["seqlens"] - s["counts"])[:, None] + t)[b, i].long()
    page = s["table"][b, at // S].long()
    for name, x, place in (("k_pages", _plain_rotate(s["k"], s["positions"], c), 0), ("v_pages", s["v"].float(), 1)):
        codes, scales = _quantise(x[b, :, i], c["kind"])
        s[name].view(torch.uint8)[page, :, at % S] = codes.view(torch.uint8)
        s["row_scales"][page, :, at % S, place] = scales[..., 0]
    k, v = _plain_read(s, T)
    return dict(q=_plain_rotate(s["q"], s["positions"], c).to(s["q"].dtype), k=k, v=v)


def _plain_accept(s):
    s["meta"].copy_(s["meta0"])
    S, (B, M), T = s["S"], s["table"].shape, s["parents"].shape[1]
    n = s["seqlens"] - s["counts"]
    t = torch.arange(T, device="cuda")
    kept = _ancestors(s["parents"], t < s["counts"][:, None]).gather(
        1, s["last"].clamp(min=0).long()[:, None, None].expand(B, 1, T))[:, 0] & (s["last"] >= 0)[:, None]
    count = kept.sum(1)
    order = torch.argsort((~kept).int(), dim=1, stable=True)  # the kept nodes, in order, first
    moves = (t < count[:, None]) & (order != t)
    from_, to = n[:, None] + order, n[:, None] + t
    rows = lambda at: s["table"].gather(1, (at // S).clamp(max=M - 1).long()) * S + at % S  # noqa: E731
    src, dst = (torch.where(moves, rows(x), -1).to(torch.int32) for x in (from_, to))
    after = n + count
    place = torch.arange(M, device="cuda") * S
    gone = (place >= after[:, None]) & (place < s["seqlens"][:, None])
    s["refs"].index_add_(0, s["table"].clamp(min=0).long().flatten(), -gone.flatten().int())
    s["table"].masked_fill_(gone, -1)
    s["seqlens"].copy_(after)
    i, j = src[moves].long(), dst[moves].long()
    for name in ("k_pages", "v_pages", "row_scales"):
        if s[name] is not None:
            x = s[name].view(torch.uint8) if s[name].dtype == torch.float8_e4m3fn else s[name]
            x[:, j // S, :, j % S] = x[:, i // S, :, i % S]
    return dict(refs=s["refs"], table=s["table"], seqlens=s["seqlens"], src=src, dst=dst, k_pages=s["k_pages"],
                v_pages=s["v_pages"], row_scales=s["row_scales"])


# -------------------------------------------------------------------------------- the package's calls
def _own(s):
    import continuous_softmax_attention_gb300 as csa

    c = s["case"]
    cache = (s["k_pages"], s["v_pages"], s["table"], s["seqlens"])
    if c["op"] == "decode":
        o, lse = csa.decode_paged(s["q"], *cache, s["k0"], s["v0"], row_scales=s["row_scales"], mode=c["mode"],
                                  workspace=s["workspace"])
        return dict(o=o, lse=lse)
    if c["op"] == "tree":
        o, lse = csa.decode_tree(s["q"], *cache, s["parents"], s["k0"], s["v0"], counts=s["counts"], row_scales=s["row_scales"],
                                 mode=c["mode"], workspace=s["workspace"])
        return dict(o=o, lse=lse)
    if c["op"] == "fill":
        q = csa.cache_append(s["k"], s["v"], *cache, row_scales=s["row_scales"], counts=s["counts"], rope=s["rope"],
                             positions=s["positions"], q=s["q"])
        k, v = csa.cache_read(*cache, c["T"], starts=s["starts"], row_scales=s["row_scales"])
        return dict(q=q, k=k, v=v)
    if c["op"] == "read":
        k, v = csa.cache_read(*cache, c["T"], starts=s["starts"], row_scales=s["row_scales"])
        return dict(k=k, v=v)
    s["meta"].copy_(s["meta0"])
    src, dst = csa.cache_accept(s["refs"], s["table"], s["seqlens"], s["S"], s["last"], c["T"], parents=s["parents"],
                                counts=s["counts"])
    csa.cache_copy_rows(s["k_pages"], s["v_pages"], src, dst, row_scales=s["row_scales"])
    return dict(refs=s["refs"], table=s["table"], seqlens=s["seqlens"], src=src, dst=dst, k_pages=s["k_pages"],
                v_pages=s["v_pages"], row_scales=s["row_scales"])


def _plain_only_read(s):
    k, v = _plain_read(s, s["case"]["T"])
    return dict(k=k, v=v)


def run(state):
    if own:
        return _own(state)
    return dict(decode=_plain_attention, tree=_plain_attention, fill=_plain_fill, read=_plain_only_read,
                accept=_plain_accept)[state["case"]["op"]](state)


# -------------------------------------------------------------------------------------------- work
def _row_bytes(case):
    """Bytes of a token's key and value in one cached head."""
    return 4 * case["d"] if case["kind"] == "bf16" else 2 * case["d"] + 8


def work(case):
    op, B, d, S, Hkv = (case[k] for k in ("op", "B", "d", "S", "Hkv"))
    row = Hkv * _row_bytes(case)
    if op == "decode":
        lens, Hq = _lens(case), case["Hq"]
        return {"bytes": sum(lens) * row + 4 * B * Hq * d + 4 * B * Hq + 4 * sum(_pages(n, S) for n in lens) + 4 * B,
                "flops": 4 * sum(lens) * Hq * d}
    if op == "tree":
        lens, (parents, counts), Hq, T = _lens(case), _trees(case), case["Hq"], case["T"]
        held = [n + c for n, c in zip(lens, counts)]
        pairs = sum(n * c + sum(len(_path(p, t)) for t in range(c)) for n, p, c in zip(lens, parents, counts))
        return {"bytes": sum(held) * row + B * Hq * T * (4 * d + 4) + 4 * sum(_pages(n, S) for n in held) + 4 * B * (T + 2),
                "flops": 4 * pairs * Hq * d}
    if op == "fill":
        size, new, T = 2 if case["dtype"] == "bf16" else 4, sum(_fill_lens(case)[1]), case["T"]
        x = B * T * case["Hq"]
        return {"bytes": 2 * x * d * size + new * Hkv * 2 * d * size + 2 * new * row + B * T * Hkv * 4 * d + 4 * len(_pairs(case)) * B * T,
                "flops": 6 * (x + new * Hkv) * sum(_pairs(case)) + 6 * new * Hkv * d}
    if op == "read":
        new = sum(min(n, case["T"]) for n in _lens(case))
        return {"bytes": new * row + B * case["T"] * Hkv * 4 * d + 4 * new // S, "flops": 2 * new * Hkv * d}
    parents, counts = _trees(case)
    paths = [_path(p, t) for p, t in zip(parents, _last(case))]
    moved = sum(u != i for path in paths for i, u in enumerate(path))
    gone = sum(_pages(n + c, S) - _pages(n + len(path), S) for n, c, path in zip(_lens(case), counts, paths))
    return {"bytes": 2 * case["L"] * moved * row + 4 * (3 * B * case["T"] + 5 * B + 2 * gone + 2 * moved), "flops": B * case["T"]}


# -------------------------------------------------------------------------------- 64-bit references
def _log_phi2(x):
    """log((e^x - 1 - x)/x^2) in 64 bits: its power series for |x| < 1/2, logarithms elsewhere."""
    small = torch.full_like(x, 1 / math.factorial(20))
    for j in range(19, 1, -1):
        small = small * x + 1 / math.factorial(j)
    far = torch.where(x.abs() < 0.5, torch.ones_like(x), x)
    up = far.clamp(min=0.5)
    above = up + torch.log1p(-(1 + up) * torch.exp(-up)) - 2 * torch.log(up)
    down = far.clamp(max=-0.5)
    below = torch.log(torch.expm1(down) - down) - 2 * torch.log(-down)
    return torch.where(x.abs() < 0.5, torch.log(small.clamp(min=1e-300)), torch.where(x > 0, above, below))


def _exact_rows(s, b, h, lo, hi):
    """Tokens lo .. hi - 1 of a sequence's cached head, in 64 bits."""
    S = s["case"]["S"]
    at = torch.arange(lo, hi, device="cuda")
    page = s["table"][b].long()[at // S]
    k, v = (s[p][page, h, at % S].double() for p in ("k_pages", "v_pages"))
    if s["row_scales"] is not None:
        scales = s["row_scales"][page, h, at % S].double()
        k, v = k * scales[:, :1], v * scales[:, 1:]
    return k, v


def _exact_attention(case, s):
    """Sequence by sequence: each row's own list of positions (the sink, the tokens before the draft, the node's path), the
    correction of each logit from its neighbours on that list, and the softmax of their sum."""
    B, Hq, Hkv, d, T = (case.get(k, 1) for k in ("B", "Hq", "Hkv", "d", "T"))
    tree = case["op"] == "tree"
    G, scale = Hq // Hkv, 1 / math.sqrt(d)
    o = torch.zeros(B, Hkv, G, T, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hkv, G, T), -math.inf, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(B, Hkv, G, T, d)
    parents, counts = _trees(case) if tree else (None, [0] * B)
    for b, n in enumerate(_lens(case)):
        c = counts[b]
        rows = c if tree else int(n > 0)
        if rows == 0:
            continue
        paths = [_path(parents[b], t) for t in range(rows)] if tree else [[]]
        deep = max(len(p) for p in paths)
        for h in range(Hkv):
            k, v = _exact_rows(s, b, h, 0, n + c)
            zero = torch.zeros(1, d, dtype=torch.float64, device="cuda")
            at = torch.tensor([p + [0] * (deep - len(p)) for p in paths], dtype=torch.int64, device="cuda").view(rows, deep) + n
            given = case["mode"] == GIVEN
            sk, sv = (s["k0"][h:h + 1].double(), s["v0"][h:h + 1].double()) if given else (zero, zero)
            sk, sv = sk.expand(rows, d), sv.expand(rows, d)
            if case["mode"] == COPY_FIRST:
                first = torch.zeros(rows, dtype=torch.int64, device="cuda") if n else at[:, 0]
                sk, sv = k[first], v[first]
            x = q[b, h, :, :rows]  # [G, rows, d]
            a = scale * torch.cat([(x * sk).sum(2, keepdim=True), x @ k[:n].T, torch.einsum("grd,rpd->grp", x, k[at])], 2)
            length = torch.tensor([1 + n + len(p) for p in paths], device="cuda")[:, None]
            place = torch.arange(a.shape[2], device="cuda")
            step = a[..., 1:] - a[..., :-1]
            gap = (place[1:] < length).expand(step.shape)
            none = torch.full_like(a[..., :1], -math.inf)
            from_next = torch.where(gap, _log_phi2(step), none)
            from_last = torch.where(gap, _log_phi2(-step), none)
            z = a + torch.logaddexp(torch.cat([none, from_last], 2), torch.cat([from_next, none], 2))
            z = torch.where(place < length, z, none)
            total = torch.logsumexp(z, 2)
            w = torch.exp(z - total[..., None])
            o[b, h, :, :rows] = w[..., :1] * sv + w[..., 1:1 + n] @ v[:n] + torch.einsum("grp,rpd->grd", w[..., 1 + n:], v[at])
            lse[b, h, :, :rows] = total
    shape = (B, Hq, T) if tree else (B, Hq)
    return dict(o=o.view(*shape, d), lse=lse.view(shape))


def _exact_rotate(x, positions, case):
    """Each pair as a complex number times e^{i angle}, one axis's pairs after the other's."""
    n, y, at = sum(_pairs(case)), x.double().clone(), 0
    for a, count in enumerate(_pairs(case)):
        pairs = torch.arange(at, at + count, device="cuda")
        angle = positions[a].double()[:, None, :, None] * torch.exp(pairs.double() * (-math.log(10000.0) / n))
        z = torch.complex(y[..., pairs], y[..., pairs + n]) * torch.polar(torch.ones_like(angle), angle)
        y[..., pairs], y[..., pairs + n] = z.real, z.imag
        at += count
    return y


def _nearest_e4m3(y):
    """y, at most 448 in magnitude, as the nearest number of 3 fraction bits and an exponent of -6 at least, ties to the even one."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    e = e - (torch.exp2(e) > y.abs()).double() * (e > -6) + (torch.exp2(e + 1) <= y.abs()).double()
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _exact_fill(case, s):
    lens, counts = _fill_lens(case)
    out = {}
    for name, x in (("k", _exact_rotate(s["k"], s["positions"], case)), ("v", s["v"].double())):
        most = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
        if case["kind"] == "e4m3":
            scale = torch.exp2(torch.floor(torch.log2(most / 448)) - 1)
            for _ in range(3):  # the logarithm may be off at a power of two
                scale = torch.where(scale * 448 < most, scale * 2, scale)
            y = _nearest_e4m3(x / scale) * scale
        else:  # what a row is scaled by is held in 32 bits
            y = torch.round(x * (127 / most).float().double()) * (most / 127).float().double()
        new = (torch.arange(case["T"], device="cuda") < _ints(counts)[:, None])[:, None, :, None]
        out[name] = torch.where(new, y, torch.zeros_like(y))
    return dict(q=_exact_rotate(s["q"], s["positions"], case), **out)


def _exact_read(case, s):
    B, T, Hkv, d = (case[k] for k in ("B", "T", "Hkv", "d"))
    out = dict(k=torch.zeros(B, Hkv, T, d, dtype=torch.float64, device="cuda"))
    out["v"] = out["k"].clone()
    for b, n in enumerate(_lens(case)):
        lo = max(0, n - T)
        for h in range(Hkv):
            out["k"][b, h, :n - lo], out["v"][b, h, :n - lo] = _exact_rows(s, b, h, lo, n)
    return out


def exact(case, seed):
    op = case["op"]
    if op == "accept":
        return None  # whole numbers and copies: compared as they are
    s = prepare(case, seed)
    return dict(decode=_exact_attention, tree=_exact_attention, fill=_exact_fill, read=_exact_read)[op](case, s)
