"""Serving operators around a paged key-value cache: the cases they are timed and compared on.

Three operators and what has to stand between them:

* ``decode``  - one decode step of continuous softmax attention over a paged cache, grouped heads
                (the cached rows are those of ``Hkv`` heads, each read by ``Hq / Hkv`` query heads);
* ``rope``    - rotary positions with several axes on queries and keys, and its backward pass;
* ``append``  - the rows of new tokens, keys rotated, written into their pages (queries rotated beside);
* ``turnover``, ``fork``, ``compact`` - the pages of the cache: freed and reserved, forked with a copy of the
                page that goes on being written, and moved together.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the calls of this
repository's package.  A case is a dict of plain values; lengths are drawn from the case's own
``lens_seed`` so that the work does not depend on the seed of the contents.
"""
import math
import random

import torch

own = False

ZERO, COPY_FIRST, GIVEN = 0, 1, 2
PAGE_LAWS = ("uniform", "log", "full")


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user, a short chat, every head with its own keys: the latency of a single small step
        dict(name="decode_one_short", op="decode", B=1, Hq=32, Hkv=32, d=128, S=16, lo=1, hi=333, law="full",
             empty=0, mode=ZERO, lens_seed=1),
        # a server's batch under continuous batching: ragged lengths over three decades, four query heads on a
        # cached head, a few slots of the batch unused
        dict(name="decode_ragged_grouped", op="decode", B=64, Hq=32, Hkv=8, d=128, S=16, lo=1, hi=8192, law="log",
             empty=5, mode=COPY_FIRST, lens_seed=2),
        # the benchmark's decode workload (16 sequences of 4096 to 8192 tokens, 32 heads) in pages of 64
        dict(name="decode_headline_paged", op="decode", B=16, Hq=32, Hkv=32, d=128, S=64, lo=4096, hi=8192,
             law="uniform", empty=0, mode=ZERO, lens_seed=6),
        # two very long documents, heads of 64 with eight queries each and given sinks: few rows, a long axis
        dict(name="decode_long_d64", op="decode", B=2, Hq=16, Hkv=2, d=64, S=256, lo=120001, hi=131071, law="uniform",
             empty=0, mode=GIVEN, lens_seed=4),
        # the queries and keys of one decode step for a batch: latency
        dict(name="rope_step", op="rope", B=64, T=1, Hq=32, Hkv=8, d=128, dtype="bf16", sections="16,24,24",
             dealt=False, adjacent=False, inverse=False, fused=True, far=1 << 20),
        # a prompt at the benchmark's length, queries and keys read out of one fused projection
        dict(name="rope_prompt", op="rope", B=1, T=8192, Hq=32, Hkv=8, d=128, dtype="bf16", sections="16,24,24",
             dealt=False, adjacent=False, inverse=False, fused=True, far=1 << 17),
        # gradients at the training shape (4 x 16 x 2048) in 32 bits, axes dealt in turn, part of each row rotated
        dict(name="rope_backward_f32", op="rope", B=4, T=2048, Hq=16, Hkv=16, d=128, dtype="f32", sections="13,17,18",
             dealt=True, adjacent=True, inverse=True, fused=False, far=1 << 14),
        # one decode step of a batch: new keys rotated into their pages, values written, queries rotated
        dict(name="append_step", op="append", B=64, T=1, Hq=32, Hkv=8, d=128, S=16, dtype="bf16", sections="16,24,24",
             past=1000, lens_seed=8),
        # ragged prompts of up to 2048 tokens filled into the cache behind what is there
        dict(name="append_prompt", op="append", B=8, T=2048, Hq=32, Hkv=8, d=128, S=64, dtype="bf16",
             sections="16,24,24", past=777, lens_seed=9),
        # between two steps: finished sequences give their pages back, every other sequence gets room for more
        dict(name="turnover", op="turnover", B=256, S=16, P=32768, lo=1, hi=2000, law="uniform", finished=17, grow=40,
             lens_seed=10),
        # beams: 48 continuations of 12 parents, pages shared, the last partly filled page of each copied
        dict(name="fork_beams", op="fork", B=64, S=64, P=1024, L=2, Hkv=8, d=128, lo=100, hi=4000, law="uniform",
             parents=12, children=48, lens_seed=11),
        # a pool at 55% use with its pages everywhere, moved together
        dict(name="compact_pool", op="compact", B=32, S=64, P=2048, L=1, Hkv=8, d=128, lo=500, hi=4000, law="uniform",
             use=0.55, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sections(rng, d):
    half = d // 2
    total = half if rng.random() < 0.5 else rng.randint(max(1, half // 3), half)
    axes = min(rng.choice([1, 2, 3, 3, 4]), total)
    cuts = sorted(rng.sample(range(1, total), axes - 1)) if axes > 1 else []
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def _pairs(case):
    """Rotated pairs of each axis, from the case's text."""
    return [int(n) for n in case["sections"].split(",")]


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "rope", "rope", "append", "turnover", "fork", "compact"])
    ls = rng.randint(0, 1 << 30)
    if op == "decode":
        d = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 3, 4, 8, 8, 32])
        G = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16, 20])
        G = max(1, min(G, 64 // Hkv))
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 131072)
        hi = max(1, min(hi, 16 * 8192 * 32 * 128 * 3 // 4 // (B * Hkv * max(d, 16 * G))))
        law = rng.choice(PAGE_LAWS)
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, d=d, S=rng.choice([8, 16, 24, 32, 48, 64, 128, 256]),
                    lo=rng.randint(1, hi) if law == "uniform" else 1, hi=hi, law=law,
                    empty=rng.randint(0, B // 3), mode=rng.choice([ZERO, COPY_FIRST, GIVEN]), lens_seed=ls)
    if op == "rope":
        d = rng.choice([32, 64, 80, 96, 128, 128, 256, 2 * rng.randint(1, 128)])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 7])
        B = rng.choice([1, 1, 2, 3, 8, 64])
        T = _log_int(rng, 1, 8192)
        T = max(1, min(T, 8192 * 40 * 128 // (B * (Hq + Hkv) * d)))
        return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    sections=_sections(rng, d), dealt=rng.random() < 0.5, adjacent=rng.random() < 0.5,
                    inverse=rng.random() < 0.4, fused=rng.random() < 0.6, far=_log_int(rng, 16, 1 << 20))
    if op == "append":
        d = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        B = _log_int(rng, 1, 64)
        T = rng.choice([1, 1, 2, _log_int(rng, 1, 2048)])
        T = max(1, min(T, 8 * 2048 * 8 * 128 // (B * Hkv * d)))
        return dict(op=op, B=B, T=T, Hq=Hkv * rng.choice([1, 2, 4, 5]), Hkv=Hkv, d=d, S=rng.choice([8, 16, 24, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), sections=_sections(rng, d), past=_log_int(rng, 1, 1000),
                    lens_seed=ls)
    if op == "turnover":
        B, S = _log_int(rng, 1, 512), rng.choice([8, 16, 24, 32, 64])
        hi = _log_int(rng, 1, 2000)
        P = B * (-(-hi // S) + 80 // S + 2) + rng.randint(0, 8192)
        return dict(op=op, B=B, S=S, P=P, lo=1, hi=hi, law=rng.choice(PAGE_LAWS), finished=rng.randint(0, B // 2),
                    grow=rng.randint(0, 80), lens_seed=ls)
    S, Hkv, d = rng.choice([8, 16, 24, 64]), rng.choice([1, 2, 8]), rng.choice([64, 128, 256])
    hi, L = _log_int(rng, 1, 2000), rng.choice([1, 1, 2, 3])
    if op == "fork":
        parents, children = rng.randint(1, 12), rng.randint(1, 48)
        B = parents + children + rng.randint(0, 9)
        P = parents * -(-hi // S) + children + rng.randint(0, 99)
        return dict(op=op, B=B, S=S, P=P, L=L, Hkv=Hkv, d=d, lo=1, hi=hi, law=rng.choice(PAGE_LAWS), parents=parents,
                    children=children, lens_seed=ls)
    B = rng.randint(1, 32)
    return dict(op=op, B=B, S=S, P=0, L=L, Hkv=Hkv, d=d, lo=1, hi=hi, law=rng.choice(PAGE_LAWS),
                use=rng.uniform(0.2, 0.95), lens_seed=ls)


def _lens(case, count=None):
    """The lengths of a case's sequences: drawn over [lo, hi] (or its logarithm, or all hi)."""
    r, n = random.Random(case["lens_seed"]), case["B"] if count is None else count
    lo, hi, law = case["lo"], case["hi"], case["law"]
    lens = [hi if law == "full" else r.randint(lo, hi) if law == "uniform" else _log_int(r, lo, hi) for _ in range(n)]
    for i in r.sample(range(n), min(case.get("empty", 0), n)):
        lens[i] = 0
    return lens


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


def _rope_spec(case):
    if not own:
        return None
    import continuous_softmax_attention_gb300 as csa

    return csa.RopeAxes(case["d"], _pairs(case), dealt=case.get("dealt", False), adjacent=case.get("adjacent", False))


def _prepare_decode(case, seed):
    g = _gen(seed)
    B, Hq, Hkv, d, S = (case[k] for k in ("B", "Hq", "Hkv", "d", "S"))
    lens = _lens(case)
    P = sum(_pages(n, S) for n in lens) + 7
    bf = dict(generator=g, device="cuda", dtype=torch.bfloat16)
    state = dict(q=torch.randn(B, Hq, d, **bf), k_pages=torch.randn(P, Hkv, S, d, **bf), v_pages=torch.randn(P, Hkv, S, d, **bf),
                 k0=torch.randn(Hkv, d, **bf), v0=torch.randn(Hkv, d, **bf), table=_tables(lens, S, P, g),
                 seqlens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if own:
        import continuous_softmax_attention_gb300 as csa

        state["workspace"] = torch.empty(csa.decode_paged_workspace_bytes(B, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    return state


def _positions(case, g):
    """Positions [A, B, T]: the first axis counts on from a far start, the others walk the rows and columns of images."""
    A, B, T = len(_pairs(case)), case["B"], case["T"]
    start = torch.randint(0, case["far"], (1, B, 1), generator=g, device="cuda")
    t = start + torch.arange(T, device="cuda")
    axes = [t, t // 37, t % 37, t % 5][:A]
    return torch.cat(axes).to(torch.int32)


def _prepare_rope(case, seed):
    g = _gen(seed)
    B, T, Hq, Hkv, d = (case[k] for k in ("B", "T", "Hq", "Hkv", "d"))
    dt = dict(generator=g, device="cuda", dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    if case["fused"]:  # one projection [B, T, heads * d] holds queries, keys and values
        x = torch.randn(B, T, Hq + 2 * Hkv, d, **dt)
        q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
    else:
        q, k = torch.randn(B, Hq, T, d, **dt), torch.randn(B, Hkv, T, d, **dt)
    return dict(q=q, k=k, positions=_positions(case, g), rope=_rope_spec(case))


def _append_lens(case):
    r = random.Random(case["lens_seed"])
    B, T = case["B"], case["T"]
    counts = [T if T == 1 else r.randint(0, T) for _ in range(B)]
    return [r.randint(0, case["past"]) + c for c in counts], counts


def _prepare_append(case, seed):
    g = _gen(seed)
    B, T, Hq, Hkv, d, S = (case[k] for k in ("B", "T", "Hq", "Hkv", "d", "S"))
    lens, counts = _append_lens(case)
    P = sum(_pages(n, S) for n in lens) + 5
    dt = dict(generator=g, device="cuda", dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    x = torch.randn(B, T, Hq + 2 * Hkv, d, **dt)
    ints = dict(dtype=torch.int32, device="cuda")
    n, c = torch.tensor(lens, **ints), torch.tensor(counts, **ints)
    t = (n - c)[None, :, None] + torch.arange(T, device="cuda")
    return dict(q=x[:, :, :Hq].transpose(1, 2), k=x[:, :, Hq:Hq + Hkv].transpose(1, 2), v=x[:, :, Hq + Hkv:].transpose(1, 2),
                k_pages=torch.randn(P, Hkv, S, d, **dt), v_pages=torch.randn(P, Hkv, S, d, **dt), table=_tables(lens, S, P, g),
                seqlens=n, counts=c, rope=_rope_spec(case),
                positions=torch.cat([t, t // 29, t % 29, t % 7][:len(_pairs(case))]).to(torch.int32).contiguous())


def _bookkeeping(refs, table, seqlens):
    """refs [P], table [B, M] and seqlens [B] as views of one buffer, and that buffer as it was: a step begins from there."""
    meta = torch.cat([refs.to(torch.int32), table.reshape(-1).to(torch.int32), seqlens.to(torch.int32)])
    P, n = refs.numel(), table.numel()
    return dict(meta=meta, meta0=meta.clone(), refs=meta[:P], table=meta[P:P + n].view(table.shape), seqlens=meta[P + n:])


def _refs(table, P):
    return torch.bincount(table[table >= 0].to(torch.int64), minlength=P)


def _prepare_turnover(case, seed):
    g = _gen(seed)
    B, S, P = case["B"], case["S"], case["P"]
    lens = _lens(case)
    table = _tables(lens, S, P, g, M=max(_pages(n, S) for n in lens) + _pages(case["grow"], S) + 1)
    r = random.Random(case["lens_seed"] + 1)
    finished = r.sample(range(B), min(case["finished"], B))
    counts = [r.randint(0, case["grow"]) for _ in range(B)]
    ints = dict(dtype=torch.int32, device="cuda")
    return dict(_bookkeeping(_refs(table, P), table, torch.tensor(lens, **ints)), finished=torch.tensor(finished, **ints),
                counts=torch.tensor(counts, **ints), S=S)


def _pools(case, P, g):
    shape = (case["L"], P, case["Hkv"], case["S"], case["d"])
    return {n: torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16) for n in ("k_pages", "v_pages")}


def _fork_pairs(case):
    r = random.Random(case["lens_seed"] + 1)
    return [r.randrange(case["parents"]) for _ in range(case["children"])], list(range(case["parents"], case["parents"] + case["children"]))


def _prepare_fork(case, seed):
    g = _gen(seed)
    B, S, P = case["B"], case["S"], case["P"]
    lens = _lens(case, case["parents"]) + [0] * (B - case["parents"])
    table = _tables(lens, S, P, g)
    pairs = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in _fork_pairs(case)]
    return dict(_bookkeeping(_refs(table, P), table, torch.tensor(lens, dtype=torch.int32, device="cuda")), **_pools(case, P, g),
                parents=pairs[0], children=pairs[1], S=S)


def _compact_pages(case):
    return case["P"] or int(sum(_pages(n, case["S"]) for n in _lens(case)) / case["use"]) + 2


def _compact_lens(case):
    """Lengths cut so that at most the wanted share of the pool is used."""
    left, out = int(_compact_pages(case) * case["use"]), []
    for n in _lens(case):
        n = max(0, min(n, left * case["S"]))
        left -= _pages(n, case["S"])
        out.append(n)
    return out


def _prepare_compact(case, seed):
    g = _gen(seed)
    lens, P = _compact_lens(case), _compact_pages(case)
    table = _tables(lens, case["S"], P, g)
    return dict(_bookkeeping(_refs(table, P), table, torch.tensor(lens, dtype=torch.int32, device="cuda")), **_pools(case, P, g),
                S=case["S"])


def prepare(case, seed):
    state = dict(decode=_prepare_decode, rope=_prepare_rope, append=_prepare_append, turnover=_prepare_turnover, fork=_prepare_fork,
                 compact=_prepare_compact)[case["op"]](case, seed)
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


def _plain_decode(s):
    c = s["case"]
    B, Hq, Hkv, d, S = (c[k] for k in ("B", "Hq", "Hkv", "d", "S"))
    G, M, n = Hq // Hkv, s["table"].shape[1], s["seqlens"]
    at = s["table"].clamp(min=0).long()
    k, v = (s[p][at].permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * S, d).float() for p in ("k_pages", "v_pages"))
    seen = (torch.arange(M * S, device="cuda") < n[:, None])[:, None, :, None]
    k, v = k.masked_fill(~seen, 0), v.masked_fill(~seen, 0)
    k0, v0 = [(x[:, :, :1] * 0, x[:, :, :1], x0.float()[None, :, None].expand(B, Hkv, 1, d))[c["mode"]]
              for x, x0 in ((k, s["k0"]), (v, s["v0"]))]
    q = s["q"].float().view(B, Hkv, G, d) * d ** -0.5
    a = torch.cat([q @ k0.transpose(2, 3), q @ k.transpose(2, 3)], 3)  # positions 0 (the sink) to M * S
    there = (torch.arange(M * S + 1, device="cuda") <= n[:, None])[:, None, None]
    m = a.masked_fill(~there, -math.inf).amax(3, keepdim=True)
    left, right = _shares(a[..., :-1], a[..., 1:], m)
    gap = there[..., 1:]  # the interval up to a position exists if the position does
    w = torch.zeros_like(a)
    w[..., :-1] += left.masked_fill(~gap, 0)
    w[..., 1:] += right.masked_fill(~gap, 0)
    l = w.sum(3)
    o = (w[..., :1] @ v0 + w[..., 1:] @ v) / l[..., None]
    none = (n == 0)[:, None, None]
    o, lse = o.masked_fill(none[..., None], 0), (m[..., 0] + torch.log(l)).masked_fill(none, -math.inf)
    return dict(o=o.reshape(B, Hq, d).to(torch.bfloat16), lse=lse.reshape(B, Hq))


def _axis_of_pair(case):
    """The axis that each rotated pair turns by: section after section, or dealt to the axes in turn."""
    left = _pairs(case)
    if not case.get("dealt"):
        return [a for a, n in enumerate(left) for _ in range(n)]
    return [a for i in range(max(left)) for a, n in enumerate(left) if i < n]


def _plain_rotate(x, positions, case, sign):
    """x [B, H, T, d] with its pairs turned by sign * position * 10000^(-i / pairs); angles in 64 bits."""
    axis = torch.tensor(_axis_of_pair(case), device="cuda")
    n = axis.numel()
    f = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / n)
    angle = (positions.double()[axis].permute(1, 2, 0) * f)[:, None]  # [B, 1, T, pairs]
    cos, sin, y = torch.cos(angle).float(), sign * torch.sin(angle).float(), x.float()
    if case.get("adjacent"):
        u, w = y[..., 0:2 * n:2], y[..., 1:2 * n:2]
        turned = torch.stack([u * cos - w * sin, u * sin + w * cos], -1).flatten(-2)
    else:
        u, w = y[..., :n], y[..., n:2 * n]
        turned = torch.cat([u * cos - w * sin, u * sin + w * cos], -1)
    return torch.cat([turned, y[..., 2 * n:]], -1).to(x.dtype)


def _plain_rope(s):
    sign = -1.0 if s["case"]["inverse"] else 1.0
    return dict(q=_plain_rotate(s["q"], s["positions"], s["case"], sign), k=_plain_rotate(s["k"], s["positions"], s["case"], sign))


def _plain_append(s):
    c = s["case"]
    T, S = c["T"], c["S"]
    t = torch.arange(T, device="cuda")
    row = (s["seqlens"] - s["counts"])[:, None] + t  # [B, T], the cache row of each new token
    b, i = torch.nonzero(t < s["counts"][:, None], as_tuple=True)
    at = row[b, i].long()
    page = s["table"][b, at // S].long()
    s["k_pages"][page, :, at % S] = _plain_rotate(s["k"], s["positions"], c, 1.0)[b, :, i]
    s["v_pages"][page, :, at % S] = s["v"][b, :, i]
    return dict(q=_plain_rotate(s["q"], s["positions"], c, 1.0), k_pages=s["k_pages"], v_pages=s["v_pages"])


def _plain_free(s, rows):
    M = s["table"].shape[1]
    gone = torch.zeros(s["table"].shape[0], dtype=torch.bool, device="cuda")
    gone[rows.long()] = True
    used = torch.arange(M, device="cuda") * s["S"] < s["seqlens"][:, None]
    hit = used & gone[:, None]
    s["refs"].index_add_(0, s["table"].clamp(min=0).long().flatten(), -hit.flatten().int())
    s["table"].masked_fill_(hit, -1)
    s["seqlens"].masked_fill_(gone, 0)


def _take(s, wanted):
    """The lowest pages that nothing holds for the true places of `wanted` [B, M], in the order of the rows."""
    free_first = torch.argsort((s["refs"] > 0).int(), stable=True).int()
    rank = torch.cumsum(wanted.flatten().int(), 0).view(wanted.shape) - 1
    return free_first[rank.clamp(min=0).long()]


def _plain_reserve(s):
    S, M, n = s["S"], s["table"].shape[1], s["seqlens"]
    place = torch.arange(M, device="cuda")
    after = n + s["counts"]
    wanted = (place * S < after[:, None]) & (place >= ((n + S - 1) // S)[:, None])
    page = _take(s, wanted)
    s["table"].copy_(torch.where(wanted, page, s["table"]))
    s["refs"].index_add_(0, page.long().flatten(), wanted.flatten().int())
    n.copy_(after)


def _plain_turnover(s):
    s["meta"].copy_(s["meta0"])
    _plain_free(s, s["finished"])
    _plain_reserve(s)
    return dict(refs=s["refs"], table=s["table"], seqlens=s["seqlens"], shortfall=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _plain_copy(s, src, dst):
    for name in ("k_pages", "v_pages"):
        s[name][:, dst.long()] = s[name][:, src.long()]


def _plain_fork(s):
    s["meta"].copy_(s["meta0"])
    S, parents, children = s["S"], s["parents"].long(), s["children"].long()
    n, rows = s["seqlens"][parents], s["table"][parents]
    partly = n % S != 0
    last = (n // S).long()
    fresh = _take(s, partly)
    src = torch.where(partly, rows.gather(1, last.clamp(max=rows.shape[1] - 1)[:, None])[:, 0], torch.full_like(n, -1))
    dst = torch.where(partly, fresh, torch.full_like(n, -1))
    place = torch.arange(rows.shape[1], device="cuda")
    whole = place < last[:, None]
    own_page = (place == last[:, None]) & partly[:, None]
    s["table"][children] = torch.where(own_page, dst[:, None], torch.where(whole, rows, torch.full_like(rows, -1)))
    s["refs"].index_add_(0, rows.clamp(min=0).long().flatten(), whole.flatten().int())
    s["refs"].index_add_(0, dst.clamp(min=0).long(), partly.int())
    s["seqlens"][children] = n
    _plain_copy(s, src[partly], dst[partly])
    return dict(refs=s["refs"], table=s["table"], seqlens=s["seqlens"], src=src, dst=dst, k_pages=s["k_pages"], v_pages=s["v_pages"])


def _plain_compact(s):
    s["meta"].copy_(s["meta0"])
    refs, P = s["refs"], s["refs"].numel()
    page, used = torch.arange(P, device="cuda"), refs > 0
    front = page < used.sum()
    src, dst = torch.nonzero(used & ~front).flatten(), torch.nonzero(~used & front).flatten()
    to = page.int()
    to[src] = dst.int()
    refs[dst] = refs[src]
    refs[src] = 0
    s["table"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()], s["table"]))
    _plain_copy(s, src, dst)
    return dict(refs=refs, table=s["table"], k_pages=s["k_pages"], v_pages=s["v_pages"],
                moved=torch.full((1,), src.numel(), dtype=torch.int32, device="cuda"))


# -------------------------------------------------------------------------------- the package's calls
def _own(s):
    import continuous_softmax_attention_gb300 as csa

    op = s["case"]["op"]
    if op == "decode":
        o, lse = csa.decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seqlens"], s["k0"], s["v0"],
                                  mode=s["case"]["mode"], workspace=s["workspace"])
        return dict(o=o, lse=lse)
    if op == "rope":
        q, k = (csa.rope_backward if s["case"]["inverse"] else csa.rope)(s["q"], s["k"], s["positions"], s["rope"])
        return dict(q=q, k=k)
    if op == "append":
        q = csa.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["seqlens"], counts=s["counts"], q=s["q"],
                             rope=s["rope"], positions=s["positions"])
        return dict(q=q, k_pages=s["k_pages"], v_pages=s["v_pages"])
    s["meta"].copy_(s["meta0"])
    books = (s["refs"], s["table"], s["seqlens"], s["S"])
    if op == "turnover":
        csa.cache_free(*books, s["finished"])
        return dict(refs=s["refs"], table=s["table"], seqlens=s["seqlens"], shortfall=csa.cache_reserve(*books, s["counts"]))
    if op == "fork":
        src, dst, _ = csa.cache_fork(*books, s["parents"], s["children"])
        csa.cache_copy_pages(s["k_pages"], s["v_pages"], src, dst)
        return dict(refs=s["refs"], table=s["table"], seqlens=s["seqlens"], src=src, dst=dst, k_pages=s["k_pages"], v_pages=s["v_pages"])
    src, dst, moved = csa.cache_compact(*books)
    csa.cache_copy_pages(s["k_pages"], s["v_pages"], src, dst, count=moved)
    return dict(refs=s["refs"], table=s["table"], k_pages=s["k_pages"], v_pages=s["v_pages"], moved=moved)


def run(state):
    if own:
        return _own(state)
    return dict(decode=_plain_decode, rope=_plain_rope, append=_plain_append, turnover=_plain_turnover, fork=_plain_fork,
                compact=_plain_compact)[state["case"]["op"]](state)


# -------------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "decode":
        lens, d, Hq, Hkv = _lens(case), case["d"], case["Hq"], case["Hkv"]
        rows, pages = sum(lens), sum(_pages(n, case["S"]) for n in lens)
        return {"bytes": 4 * rows * Hkv * d + 4 * case["B"] * Hq * d + 4 * case["B"] * Hq + 4 * pages + 4 * case["B"],
                "flops": 4 * rows * Hq * d}
    if op == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        x, n = case["B"] * case["T"] * (case["Hq"] + case["Hkv"]), 2 * sum(_pairs(case))
        return {"bytes": 2 * x * case["d"] * size + 4 * len(_pairs(case)) * case["B"] * case["T"], "flops": 3 * x * n}
    if op == "append":
        size = 2 if case["dtype"] == "bf16" else 4
        new, d = sum(_append_lens(case)[1]), case["d"]
        x = case["B"] * case["T"] * case["Hq"]
        return {"bytes": 2 * (x + 2 * new * case["Hkv"]) * d * size + 4 * len(_pairs(case)) * case["B"] * case["T"],
                "flops": 6 * (x + new * case["Hkv"]) * sum(_pairs(case))}
    B, S = case["B"], case["S"]
    if op == "turnover":
        lens = _lens(case)
        r = random.Random(case["lens_seed"] + 1)
        r.sample(range(B), min(case["finished"], B))
        new = sum(_pages(n + r.randint(0, case["grow"]), S) - _pages(n, S) for n in lens)
        gone = case["finished"] * _pages((case["lo"] + case["hi"]) // 2, S)
        return {"bytes": 4 * (case["P"] + 3 * B + 3 * gone + 2 * new), "flops": case["P"]}
    page = 2 * 2 * case["L"] * case["Hkv"] * S * case["d"]  # keys and values of one page, in every layer
    if op == "fork":
        lens = _lens(case, case["parents"])
        parents, _ = _fork_pairs(case)
        moved, shared = sum(lens[p] % S != 0 for p in parents), sum(_pages(lens[p], S) for p in parents)
        return {"bytes": 2 * moved * page + 4 * (case["P"] + 4 * shared), "flops": shared}
    P, used = _compact_pages(case), sum(_pages(n, S) for n in _compact_lens(case))
    moved = used * (P - used) // P
    return {"bytes": 2 * moved * page + 4 * (P + 2 * moved + 2 * used), "flops": P}


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


def _exact_decode(case, s):
    """Row by row: logits, the correction of each from its neighbours, and the softmax of their sum."""
    B, Hq, Hkv, d, S = (case[k] for k in ("B", "Hq", "Hkv", "d", "S"))
    G, scale = Hq // Hkv, 1 / math.sqrt(d)
    o = torch.zeros(B, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        ids = s["table"][b, :_pages(n, S)].long()
        for h in range(Hkv):
            k, v = (s[p][ids, h].reshape(-1, d)[:n].double() for p in ("k_pages", "v_pages"))
            first = {ZERO: (k[:1] * 0, v[:1] * 0), COPY_FIRST: (k[:1], v[:1]),
                     GIVEN: (s["k0"][h:h + 1].double(), s["v0"][h:h + 1].double())}[case["mode"]]
            k, v = torch.cat([first[0], k]), torch.cat([first[1], v])
            a = scale * s["q"][b, h * G:(h + 1) * G].double() @ k.T
            step = a[:, 1:] - a[:, :-1]
            none = torch.full_like(a[:, :1], -math.inf)
            z = a + torch.logaddexp(torch.cat([none, _log_phi2(-step)], 1), torch.cat([_log_phi2(step), none], 1))
            total = torch.logsumexp(z, 1)
            o[b, h * G:(h + 1) * G] = torch.exp(z - total[:, None]) @ v
            lse[b, h * G:(h + 1) * G] = total
    return dict(o=o, lse=lse)


def _exact_rotate(x, positions, case, sign):
    """Each pair as a complex number times e^{i angle}, one axis's pairs after the other's."""
    axis = _axis_of_pair(case)
    n = len(axis)
    y = x.double().clone()
    for a in range(len(_pairs(case))):
        pairs = torch.tensor([i for i in range(n) if axis[i] == a], device="cuda")
        re, im = (2 * pairs, 2 * pairs + 1) if case.get("adjacent") else (pairs, pairs + n)
        angle = sign * positions[a].double()[:, None, :, None] * torch.exp(pairs.double() * (-math.log(10000.0) / n))
        z = torch.complex(y[..., re], y[..., im]) * torch.polar(torch.ones_like(angle), angle)
        y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_append(case, s):
    lens, counts = _append_lens(case)
    k = _exact_rotate(s["k"], s["positions"], case, 1.0)
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    for b, (n, c) in enumerate(zip(lens, counts)):
        rows = torch.arange(n - c, n, device="cuda")
        page = s["table"][b].long()[rows // case["S"]]
        kp[page, :, rows % case["S"]] = k[b, :, :c].transpose(0, 1)
        vp[page, :, rows % case["S"]] = s["v"][b, :, :c].double().transpose(0, 1)
    return dict(q=_exact_rotate(s["q"], s["positions"], case, 1.0), k_pages=kp, v_pages=vp)


def exact(case, seed):
    op = case["op"]
    if op not in ("decode", "rope", "append"):
        return None  # whole numbers and copies: compared as they are
    s = prepare(case, seed)
    if op == "decode":
        return _exact_decode(case, s)
    if op == "append":
        return _exact_append(case, s)
    sign = -1.0 if case["inverse"] else 1.0
    return dict(q=_exact_rotate(s["q"], s["positions"], case, sign), k=_exact_rotate(s["k"], s["positions"], case, sign))
