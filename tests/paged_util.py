"""Helpers of the paged-cache tests: scattered pages, a host model of the page
bookkeeping, rotary positions in extended precision, and error bounds.

Bounds.  A result rounded once to a type of half step u (2^-8 bf16, 2^-24 fp32)
is within u |ref| of the reference plus the error of its fp32 arithmetic.  For
the decode step that arithmetic is: logits of d products summed in fp32, off by
at most (d + 4) 2^-24 A with A = scale * max_i sum_c |q_c k_ic| (the 4 covers
the scale's and the exponent's own roundings); weights that are exponentials of
these, so off by that much relative, plus 2^-16 for the weight function and for
the rounding of the weights to a sum of two bf16 numbers.  Numerator and
denominator are both off by that, so o is off by at most twice it times
max |v|, and lse by it once."""
import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def pages_of(n, S):
    return -(-n // S)


def scattered(lens, S, P, seed, M=None):
    """A block table with the sequences' pages drawn from a permuted pool; entries
    behind a sequence's pages are out of range on purpose (they are never read)."""
    M = max([pages_of(n, S) for n in lens] + [1]) if M is None else M
    order = np.random.default_rng(seed).permutation(P)
    table, at = np.full((len(lens), M), -77, np.int32), 0
    for b, n in enumerate(lens):
        k = pages_of(n, S)
        table[b, :k] = order[at:at + k]
        at += k
    return table


def rows_of(pages, table_row, n, S):
    """The first n rows [Hkv, n, d] of a sequence out of its pages."""
    ids = torch.as_tensor(table_row[:pages_of(n, S)].astype(np.int64))
    x = pages[ids]  # [k, Hkv, S, d]
    return x.permute(1, 0, 2, 3).reshape(pages.shape[1], -1, pages.shape[3])[:, :n]


def decode_bounds(q, k, v, ref_o, ref_lse, scale):
    """Bounds on |o - ref_o| and |lse - ref_lse| for one (sequence, head): q [d],
    k, v [n + 1, d] with the sink's pair, ref_o [d]."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    a = abs(scale) * (np.abs(k) @ np.abs(q)).max()
    rel = (q.size + 4) * 2.0 ** -24 * a + 2.0 ** -16
    return (HALF_STEP[torch.bfloat16] * np.abs(ref_o) + 2 * rel * np.abs(v).max(),
            rel + 2.0 ** -22 * (1 + abs(ref_lse)))


class Books:
    """The page bookkeeping on the host, one sequence and page at a time."""

    def __init__(self, B, P, S, M):
        self.S, self.M, self.P = S, M, P
        self.refs, self.table, self.lens = [0] * P, [[-1] * M for _ in range(B)], [0] * B

    def lowest(self, count):
        free = [p for p in range(self.P) if self.refs[p] == 0]
        return free[:count], max(0, count - len(free))

    def reserve(self, counts):
        if any(c < 0 or n + c > self.M * self.S for n, c in zip(self.lens, counts)):
            return -1
        need = [pages_of(n + c, self.S) - pages_of(n, self.S) for n, c in zip(self.lens, counts)]
        got, short = self.lowest(sum(need))
        if short:
            return short
        for b, c in enumerate(counts):
            for j in range(need[b]):
                page = got.pop(0)
                self.refs[page] = 1
                self.table[b][pages_of(self.lens[b], self.S) + j] = page
            self.lens[b] += c
        return 0

    def free(self, rows):
        if any(r < -1 or r >= len(self.lens) for r in rows):
            return
        for r in dict.fromkeys(r for r in rows if r >= 0):
            for j in range(pages_of(self.lens[r], self.S)):
                self.refs[self.table[r][j]] -= 1
                self.table[r][j] = -1
            self.lens[r] = 0

    def fork(self, parents, children):
        n, B = len(parents), len(self.lens)
        none = [-1] * n
        pairs = [(i, p, c) for i, (p, c) in enumerate(zip(parents, children)) if p >= 0 and c >= 0]
        kids = [c for _, _, c in pairs]
        if any(p >= B or c >= B for _, p, c in pairs) or len(set(kids)) < len(kids) or any(self.lens[c] for c in kids):
            return none, none, -1
        before = list(self.lens)
        got, short = self.lowest(sum(before[p] % self.S != 0 for _, p, _ in pairs))
        if short:
            return none, none, short
        src, dst = list(none), list(none)
        for i, p, c in pairs:
            whole = before[p] // self.S
            row = self.table[p][:whole]
            for page in row:
                self.refs[page] += 1
            if before[p] % self.S:
                src[i], dst[i] = self.table[p][whole], got.pop(0)
                self.refs[dst[i]] = 1
                row = row + [dst[i]]
            self.table[c] = row + [-1] * (self.M - len(row))
            self.lens[c] = before[p]
        return src, dst, 0

    def compact(self):
        U = sum(r > 0 for r in self.refs)
        src = [p for p in range(U, self.P) if self.refs[p] > 0]
        dst = [p for p in range(U) if self.refs[p] == 0]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        for b, n in enumerate(self.lens):
            for j in range(pages_of(n, self.S)):
                self.table[b][j] = to.get(self.table[b][j], self.table[b][j])
        return src, dst


def axis_of_pairs(sections, dealt):
    if not dealt:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    out, left = [], list(sections)
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def rotated(x, positions, sections, *, base=10000.0, adjacent=False, dealt=False, inverse=False):
    """x [B, H, T, d] (any float tensor) turned in 64 bits; positions [A, B, T].
    Angles are reduced in long double, so far positions keep them."""
    x = x.detach().cpu().double().numpy().copy()
    axis = axis_of_pairs(sections, dealt)
    n = len(axis)
    pos = np.asarray(positions.cpu() if torch.is_tensor(positions) else positions)
    two_pi = np.longdouble("6.283185307179586476925286766559")
    for i, a in enumerate(axis):
        f = np.power(np.longdouble(base), -np.longdouble(i) / n) / two_pi
        turns = pos[a].astype(np.longdouble) * f
        ang = ((turns - np.floor(turns)) * two_pi).astype(np.float64)[:, None]
        c, s = np.cos(ang), np.sin(ang) * (-1 if inverse else 1)
        iu, iw = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
        u, w = x[..., iu].copy(), x[..., iw].copy()
        x[..., iu], x[..., iw] = u * c - w * s, u * s + w * c
    return x


def rope_bound(x, ref):
    """One rounding of the result; in fp32 before it, sine and cosine within 4
    steps of 2^-24 absolute (the angle's rounding to fp32, pi 2^-24 at most, and
    the function's own) and two roundings of products and sum."""
    dt, big = x.dtype, x.detach().abs().max().item()
    return HALF_STEP[dt] * np.abs(ref) + 2 * (4 + 2) * 2.0 ** -24 * big
