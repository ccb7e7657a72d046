"""The paged cache and rotary positions of libcsa.so (include/csa.h, "Paged
key-value caches" and csa_rope_plan) on torch tensors.

Signatures and documentation; the checks of the arguments and the calls are in
csrc/csa_torch.cpp (module _csa_torch, built beside libcsa.so).  Every call
runs on the device of its tensors and is asynchronous on torch's current
stream there, or on ``stream``; what it allocates (outputs, workspaces)
belongs to that stream.  Outside autograd, as the rest of the package: results
have no history, also where an input requires a gradient (rope_backward gives
it).  What a call writes gets a new version, so that autograd refuses to go
backward through a saved tensor that was overwritten.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import CSA_ERR_UNSUPPORTED, CsaError, _check, load

MAX_PAIRS, MAX_AXES = 128, 8
_FLAG_ADJACENT, _FLAG_DEALT = 1, 2


class _Unloaded:
    """Stands for _csa_torch until the first call, and raises if it has not
    been built: there is no other path."""

    def __getattr__(self, name):
        global _native
        load()  # libcsa.so, with the message if it is missing
        try:
            from . import _csa_torch
        except ImportError as e:
            raise RuntimeError("_csa_torch is missing or does not fit this torch: build it with "
                               "`python -m continuous_softmax_attention_gb300.build`") from e
        _csa_torch.set_error(_lib.CsaError)
        _native = _csa_torch
        return getattr(_native, name)


_native = _Unloaded()


def _there(fn, params):
    """fn(**params) with params' stream as the current one."""
    stream = params.pop("stream")
    with torch.cuda.stream(stream):
        first = next(iter(params.values()))
        if isinstance(first, torch.Tensor) and first.device != stream.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {first.device}")
        return fn(**params)


class _Plan(ctypes.Structure):
    """csa_rope_plan."""

    _fields_ = [("pairs", ctypes.c_int), ("axes", ctypes.c_int), ("adjacent", ctypes.c_int),
                ("axis", ctypes.c_ubyte * MAX_PAIRS), ("turn", ctypes.c_ulonglong * MAX_PAIRS)]


class RopeAxes:
    """Rotary positions with several axes: the plan that rope, rope_backward
    and cache_append take.

    d: row length; sections: how many pairs of a row turn by each axis (one to
    eight axes, n = sum(sections) <= d / 2 pairs); pair i turns by
    position * base^(-i / n).  adjacent: pairs (2i, 2i + 1) instead of
    (i, i + n).  dealt: pairs dealt to the axes in turn instead of section
    after section.  Columns from 2n on are left as they are."""

    def __init__(self, d: int, sections, *, base: float = 10000.0, adjacent: bool = False,
                 dealt: bool = False):
        sections = [int(s) for s in sections]
        if not 1 <= len(sections) <= MAX_AXES or min(sections) < 0 or sum(sections) < 1:
            raise ValueError("sections: one to eight counts of pairs, not all 0")
        if 2 * sum(sections) > d or d > 2 * MAX_PAIRS:
            raise ValueError(f"{sum(sections)} pairs do not fit a row of {d} (at most "
                             f"{2 * MAX_PAIRS} columns)")
        self.d, self.sections, self.base = int(d), tuple(sections), float(base)
        self.adjacent, self.dealt, self.axes = bool(adjacent), bool(dealt), len(sections)
        self._plan = _Plan()
        flags = (_FLAG_ADJACENT if adjacent else 0) | (_FLAG_DEALT if dealt else 0)
        _check(load().csa_rope_plan_init(ctypes.byref(self._plan), (ctypes.c_int * self.axes)(*sections),
                                         self.axes, self.base, flags), "csa_rope_plan_init")
        self._at = ctypes.addressof(self._plan)  # lives as long as this object


def _need_plan(plan):
    if not isinstance(plan, RopeAxes):
        raise ValueError("the plan must be a RopeAxes")


def decode_paged_workspace_bytes(B: int, Hq: int, Hkv: int, d: int) -> int:
    """Bytes of workspace csa_decode_paged needs (host-side, no device needed)."""
    n = int(load().csa_decode_paged_workspace_bytes(int(B), int(Hq), int(Hkv), int(d)))
    if n < 0:
        raise CsaError(CSA_ERR_UNSUPPORTED, "csa_decode_paged_workspace_bytes")
    return n


def decode_paged(q, k_pages, v_pages, block_table, seqlens, k0=None, v0=None, *, mode: int = 0,
                 scale=None, out=None, lse=None, workspace=None, want_lse: bool = True,
                 stream=None):
    """One decode step over a paged cache: the newest token of each sequence
    against the rows in its pages.  Returns (o [B, Hq, d], lse [B, Hq]).

    q: bf16 CUDA [B, Hq, d]; k_pages, v_pages: bf16 [P, Hkv, S, d], query head
    h reading cached head h // (Hq // Hkv); block_table: int32 [B, M], the
    pages of each sequence in order; seqlens: int32 [B], the tokens held with
    the newest one (0: an empty place in the batch, o = 0 and lse = -inf).
    k0, v0: [Hkv, d] in mode GIVEN (2).  d in {64, 128, 256}, S a multiple of
    8.  workspace: a CUDA tensor of decode_paged_workspace_bytes(B, Hq, Hkv,
    d) bytes (allocated when None); stream: as everywhere, torch's current
    stream when None."""
    if stream is not None:
        return _there(decode_paged, locals())
    return _native.decode_paged(q, k_pages, v_pages, block_table, seqlens, k0, v0, mode, scale, out, lse,
                                workspace, want_lse)


# ------------------------------------------------------------ rotary positions
def rope(q, k, positions, plan, *, q_out=None, k_out=None, stream=None):
    """Rotary positions on queries and keys.  Returns (q', k').

    q: CUDA [B, Hq, T, d], k: [B, Hkv, T, d] or None, both bf16 or both fp32,
    with any strides whose last one is 1 (for instance slices of one fused
    projection); positions: int32 [axes, B, T] of any strides ([B, T] or [T]
    too for a plan of one axis); plan: a RopeAxes.  q_out, k_out: where the
    results go (contiguous tensors when None); each may be its own input, and
    overlaps no input otherwise."""
    if stream is not None:
        return _there(rope, locals())
    _need_plan(plan)
    return _native.rope(q, k, positions, plan._at, plan.d, q_out, k_out, 0)


def rope_backward(dq, dk, positions, plan, *, q_out=None, k_out=None, stream=None):
    """Backward pass of rope: the gradients of q and k from the gradients of
    rope's results, rotated by the negative angles.  Arguments as rope."""
    if stream is not None:
        return _there(rope_backward, locals())
    _need_plan(plan)
    return _native.rope(dq, dk, positions, plan._at, plan.d, q_out, k_out, 1)


def cache_append(k, v, k_pages, v_pages, block_table, seqlens, *, counts=None, rope=None,
                 positions=None, q=None, q_out=None, stream=None):
    """Writes the rows of new tokens into their pages, the keys rotated if a
    plan is given, and rotates their queries beside.  Returns q' (None without q).

    k, v: CUDA [B, Hkv, T, d] of any strides whose last one is 1, bf16 or
    fp32; row t < counts[b] (int32 [B]; T each when None) becomes token
    seqlens[b] - counts[b] + t of sequence b: seqlens counts the new tokens
    already, as cache_reserve leaves it.  k_pages, v_pages: [P, Hkv, S, d];
    block_table: int32 [B, M].  rope: a RopeAxes; positions as in rope(), or
    None for a token's place in the cache.  q: [B, Hq, T, d], with rope only.
    decode_paged reads bf16 pools; fp32 ones are for a caller's own attention,
    and so is attention of a prompt's rows over the pages behind a past: the
    calls here attend from one new token per sequence."""
    if stream is not None:
        return _there(cache_append, locals())
    if rope is None:
        return _native.cache_append(k, v, k_pages, v_pages, block_table, seqlens, counts, None, 0, positions, q,
                                    q_out)
    _need_plan(rope)
    return _native.cache_append(k, v, k_pages, v_pages, block_table, seqlens, counts, rope._at, rope.d, positions,
                                q, q_out)


# ------------------------------------------------------------------------ pages
def cache_reserve(page_refs, block_table, seqlens, page_size: int, counts, *, shortfall=None,
                  stream=None):
    """Room for counts[b] more tokens of every sequence: takes the missing pages
    (lowest-numbered free ones first), enters them into the table and adds
    counts to seqlens.  Returns shortfall (int32 [1], on the device): 0 if it
    was done, else nothing has changed and it is the number of pages missing
    from the pool, or -1 for a count that does not fit the table.

    page_refs: int32 [P]; block_table: int32 [B, M]; seqlens, counts: int32 [B]."""
    if stream is not None:
        return _there(cache_reserve, locals())
    return _native.cache_reserve(page_refs, block_table, seqlens, page_size, counts, shortfall)


def cache_free(page_refs, block_table, seqlens, page_size: int, rows, *, stream=None):
    """The listed sequences (int32 [R]; -1 is padding) give their pages back:
    their entries become -1, their lengths 0."""
    if stream is not None:
        return _there(cache_free, locals())
    return _native.cache_free(page_refs, block_table, seqlens, page_size, rows)


def cache_fork(page_refs, block_table, seqlens, page_size: int, parents, children, *, stream=None):
    """children[i] (an empty sequence) becomes a copy of parents[i] (int32 [n]
    both, n <= 4096; a negative entry is padding): full pages are shared, a
    partly filled last page gets a page of its own.  Returns (src, dst,
    shortfall): the pages to copy with cache_copy_pages in every pool (-1
    where there is none), and shortfall as in cache_reserve."""
    if stream is not None:
        return _there(cache_fork, locals())
    return _native.cache_fork(page_refs, block_table, seqlens, page_size, parents, children)


def cache_compact(page_refs, block_table, seqlens, page_size: int, *, stream=None):
    """Gives the U held pages the numbers 0 .. U - 1.  Returns (src, dst,
    moved): int32 [P // 2] twice and [1]; the pools follow with
    cache_copy_pages(..., src, dst, count=moved) before they are read again."""
    if stream is not None:
        return _there(cache_compact, locals())
    return _native.cache_compact(page_refs, block_table, seqlens, page_size)


def cache_copy_pages(k_pages, v_pages, src, dst, *, count=None, stream=None):
    """Copies page src[i] onto page dst[i] (int32 [n]; a negative entry is
    padding) for i < min(n, count) in both pools, [P, Hkv, S, d] or, for
    several layers at once, [L, P, Hkv, S, d]; any type.  v_pages may be None;
    count: int32 [1] on the device.  A page that is a dst must not occur in
    another pair."""
    if stream is not None:
        return _there(cache_copy_pages, locals())
    return _native.cache_copy_pages(k_pages, v_pages, src, dst, count)
