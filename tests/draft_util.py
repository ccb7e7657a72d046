"""Helpers of the tests of 8-bit caches and drafted tokens: rows quantised and trees
accepted on the host, one value and one sequence at a time.

Numbers of 8 bits.  An e4m3 number is off by at most half a step, 2^-4 of the value
or 2^-10 where it is below 2^-6; an int8 code by half. With a scale s these are 2^-4 |x|
or 2^-10 s, and s / 2. The int8 scale max / 127 and the factor 127 / max are each rounded
to fp32, 2^-24 relative, and a code's product with either is 127 s at most: 127 s * 2^-24
more for each of them, and for a product rounded to fp32, so s / 2 (1 + 3 * 254 * 2^-24),
less than s / 2 (1 + 2^-14)."""
import math

import numpy as np
import torch

from paged_util import Books, pages_of

KINDS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def nearest_e4m3(y):
    """|y| <= 448 to the nearest multiple of its step, ties to even."""
    y = np.asarray(y, np.float64)
    e = np.maximum(np.frexp(y)[1] - 1, -6)
    step = np.ldexp(1.0, e - 3)
    return np.rint(y / step) * step  # a carry into the next exponent is exact


def scale_of(most, kind):
    """The scale of a row with the largest magnitude `most` (fp32), elementwise; 0 where the row is held as zeros."""
    most = np.asarray(most, np.float32)
    out = np.zeros(most.shape, np.float32)
    for i in np.ndindex(most.shape):
        if most[i] < 2.0 ** -100:
            continue
        if kind == "int8":
            out[i] = np.float32(most[i] / np.float32(127))
        else:
            e = -140
            while math.ldexp(448.0, e) < most[i]:
                e += 1
            out[i] = math.ldexp(1.0, e)
    return out


def quantised(x, kind):
    """(code values, scales) of rows x [..., d], finite."""
    x = np.asarray(x, np.float64)
    most = np.abs(x).max(-1).astype(np.float32)
    s = scale_of(most, kind)
    none = (s == 0)[..., None]
    if kind == "e4m3":
        c = nearest_e4m3(np.where(none, 0, x) / np.where(s > 0, s, 1)[..., None].astype(np.float64))
    else:
        factor = np.float32(127) / np.where(s > 0, most, 1).astype(np.float32)
        c = np.rint(np.where(none, 0, x) * factor[..., None].astype(np.float64))
    return c, s


def half_step(x, s, kind):
    """How far a quantised value may be from x."""
    x, s = np.abs(np.asarray(x, np.float64)), np.asarray(s, np.float64)[..., None]
    return np.maximum(2.0 ** -4 * x, 2.0 ** -10 * s) if kind == "e4m3" else 0.5 * s * (1 + 2.0 ** -14)


def random_pools(P, H, S, d, kind, g, spread=1.0):
    """k_pages, v_pages and row_scales (None for bf16) of random rows."""
    if kind == "bf16":
        return torch.randn(P, H, S, d, generator=g).to(torch.bfloat16), torch.randn(P, H, S, d, generator=g).to(torch.bfloat16), None
    pools = []
    for _ in range(2):
        c = torch.randn(P, H, S, d, generator=g)
        pools.append((c * 100).clamp(-448, 448).to(torch.float8_e4m3fn) if kind == "e4m3" else (c * 40).clamp(-127, 127).to(torch.int8))
    scales = torch.exp2(torch.randn(P, H, S, 2, generator=g) * spread) * (0.01 if kind == "e4m3" else 0.025)
    return pools[0], pools[1], scales


def values(k, v, scales):
    """The pools' values in 64 bits."""
    if scales is None:
        return k.double(), v.double()
    return k.float().double() * scales[..., :1].double(), v.float().double() * scales[..., 1:].double()


def path_of(parents, node):
    path = []
    while node >= 0:
        path.append(node)
        node = parents[node]
    return path[::-1]


def tree(T, kind, rng):
    """Parents of T nodes: "chain", "star" (all begin anew), "wide" (four children each) or "random"."""
    if kind == "chain":
        return list(range(-1, T - 1))
    if kind == "star":
        return [-1] * T
    if kind == "wide":
        return [-1 if t == 0 else (t - 1) // 4 for t in range(T)]
    return [-1 if t == 0 or rng.random() < 0.15 else int(rng.integers(max(0, t - 7), t)) for t in range(T)]


class DraftBooks(Books):
    """Books with the accepted branch of a draft kept."""

    def accept(self, parents, counts, last, T):
        src, dst = [[-1] * T for _ in self.lens], [[-1] * T for _ in self.lens]
        for b, (c, leaf) in enumerate(zip(counts, last)):
            n, held = self.lens[b] - c, self.lens[b]
            path = path_of(parents[b], leaf)
            row = lambda at: self.table[b][at // self.S] * self.S + at % self.S  # noqa: E731
            for i, u in enumerate(path):
                if u != i:
                    src[b][i], dst[b][i] = row(n + u), row(n + i)
            self.lens[b] = n + len(path)
            for j in range(pages_of(self.lens[b], self.S), pages_of(held, self.S)):
                self.refs[self.table[b][j]] -= 1
                self.table[b][j] = -1
        return src, dst


def bounds(q, k, v, ref_o, ref_lse, scale, weights):
    """Bounds on |o - ref_o| and |lse - ref_lse| of one row: q [d], k, v [n + 1, d] with the sink's pair, in 64 bits.
    As paged_util.decode_bounds: logits off by (d + 8) 2^-24 A, weights by that and 2^-16 for the weight function, o by
    twice it times max |v|.  Then `weights`, the rounding of the weights to 16 bits: it moves the numerator alone, by at
    most that much of max |v|."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    a = abs(scale) * (np.abs(k) @ np.abs(q)).max()
    rel = (q.size + 8) * 2.0 ** -24 * a + 2.0 ** -16
    return (2.0 ** -8 * np.abs(ref_o) + (2 * rel + weights) * np.abs(v).max(), rel + 2.0 ** -22 * (1 + abs(ref_lse)))


def bounds8(q, k, v, ref_o, ref_lse, scale):
    """The same over 8-bit pools, weights as single fp16 numbers: 2^-11 relative, or 2^-25 absolute where they are below
    2^-14.  They are weights times a value's scale by a power of two (at most twice the largest scale) times 2^7, so the
    absolute part moves o by at most 2^-32 of 448 * twice the largest scale per row, over the sum of the weights.  448 scales
    are at most 4 max |v| here, and the weight of the largest logit alone is at least 2^-4 for steps below 16: 2^-26 max |v|
    for each row."""
    return bounds(q, k, v, ref_o, ref_lse, scale, 2.0 ** -11 + len(k) * 2.0 ** -26)


def bounds_tree(kind, rows, q, k, v, ref_o, ref_lse, scale):
    """A row of a tree, `rows` = T times the query heads on a cached head.  Weights over bf16 pools are two bf16 numbers
    (2^-16), over 8-bit ones as bounds8.  Above 16 rows an interval's integral is divided between its two rows within 4e-4 < 2^-11 of the smaller share (the error of the quotients is relative
    to the left share, and the right one is the rest): that moves the numerator by at most 4e-4 times the share times the
    difference of two values, in all by at most 2 * 4e-4 / 2 max |v|, since the smaller shares are at most half of the sum."""
    if kind != "bf16":
        if rows <= 16:
            return bounds8(q, k, v, ref_o, ref_lse, scale)
        return bounds(q, k, v, ref_o, ref_lse, scale, 2.0 ** -10 + len(k) * 2.0 ** -26)
    return bounds(q, k, v, ref_o, ref_lse, scale, 2.0 ** -16 + (2.0 ** -11 if rows > 16 else 0.0))
