"""ctypes binding of libcsa.so's paged cache and rotary positions
(include/csa.h, "Paged key-value caches" and csa_rope_plan).

Argument marshalling only, as in _lib.py.  Every call runs on the device of
its tensors and is asynchronous on torch's current stream there, or on
``stream``; what it allocates (outputs, workspaces) belongs to that stream.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import CSA_ERR_UNSUPPORTED, CsaError, _check, _check_tensor, load

MAX_PAIRS, MAX_AXES = 128, 8
_FLAG_ADJACENT, _FLAG_DEALT = 1, 2


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
        self._ref = ctypes.byref(self._plan)


_current_device = torch.cuda.current_device
# the handle of the current stream; torch.cuda.current_stream() costs 3 us here, as much as a launch
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _there(fn, params, first):
    """fn(**params) on the device of `first` and on params' stream."""
    stream, dev = params.pop("stream"), first.device
    if dev.type != "cuda":
        raise ValueError(f"{fn.__name__} takes CUDA tensors")
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.device(dev):
        if stream is None:
            return fn(**params)
        with torch.cuda.stream(stream):
            return fn(**params)


def _need(t, name, dtype, shape, dev):
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _check_tensor(t, name, dtype, shape, dev)


def _at(t):
    return None if t is None else t.data_ptr()


def _workspace(workspace, nbytes, dev):
    if workspace is None:
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace


def _out(t, name, dtype, shape, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _need(t, name, dtype, shape, dev)
    return t


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
    if stream is not None or q.device.index is None or q.device.index != _current_device():
        return _there(decode_paged, locals(), q)
    if q.dim() != 3 or k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q is [B, Hq, d], the pools [P, Hkv, S, d], block_table [B, M]")
    B, Hq, d = q.shape
    P, Hkv, S, _ = k_pages.shape
    M = block_table.shape[1]
    dev, bf = q.device, torch.bfloat16
    _need(q, "q", bf, (B, Hq, d), dev)
    _need(k_pages, "k_pages", bf, (P, Hkv, S, d), dev)
    _need(v_pages, "v_pages", bf, (P, Hkv, S, d), dev)
    _need(block_table, "block_table", torch.int32, (B, M), dev)
    _need(seqlens, "seqlens", torch.int32, (B,), dev)
    if mode == 2:
        if k0 is None or v0 is None:
            raise ValueError("mode 2 (given sink) needs k0 and v0")
        _need(k0, "k0", bf, (Hkv, d), dev)
        _need(v0, "v0", bf, (Hkv, d), dev)
    else:
        k0 = v0 = None
    if scale is None:
        scale = 1.0 / d ** 0.5
    out = _out(out, "out", bf, (B, Hq, d), dev)
    if lse is not None or want_lse:
        lse = _out(lse, "lse", torch.float32, (B, Hq), dev)
    lib = load()
    if workspace is None:
        workspace = _workspace(None, max(0, lib.csa_decode_paged_workspace_bytes(B, Hq, Hkv, d)), dev)
    else:
        _workspace(workspace, 0, dev)
    _check(lib.csa_decode_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _at(k0), _at(v0), block_table.data_ptr(),
                                seqlens.data_ptr(), out.data_ptr(), _at(lse), workspace.data_ptr(), workspace.nbytes, B, Hq,
                                Hkv, P, S, M, d, scale, mode, _raw_stream(dev.index)), "csa_decode_paged")
    return out, lse


# ------------------------------------------------------------ rotary positions
_Strides = ctypes.c_longlong * 3


def _rows(t, name, dtype, shape, dev, written=False):
    """Checks a tensor of rows [B, H, T, d] of any strides and returns its
    strides over batch, head and time (None if it is contiguous)."""
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return None
    sb, sh, st, sd = t.stride()
    if sd != 1 and shape[3] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if written:
        reach = shape[3]
        for stride, size in sorted(zip((sb, sh, st), shape)):
            if size > 1:
                if stride < reach:
                    raise ValueError(f"rows of {name} overlap")
                reach += stride * (size - 1)
    return _Strides(sb, sh, st)


def _position_strides(positions, plan, B, T, dev):
    if positions.device != dev or positions.dtype is not torch.int32:
        raise ValueError(f"positions must be int32 on {dev}, got {positions.dtype} on {positions.device}")
    shape = positions.shape
    if shape == (plan.axes, B, T):
        return None if positions.is_contiguous() else _Strides(*positions.stride())
    if plan.axes == 1 and shape == (B, T):
        return _Strides(0, *positions.stride())
    if plan.axes == 1 and shape == (T,):
        return _Strides(0, 0, *positions.stride())
    raise ValueError(f"positions must have shape {(plan.axes, B, T)}"
                     + (f", {(B, T)} or {(T,)}" if plan.axes == 1 else "") + f", got {tuple(shape)}")


def _check_plan(plan, d):
    if not isinstance(plan, RopeAxes):
        raise ValueError("the plan must be a RopeAxes")
    if plan.d != d:
        raise ValueError(f"the plan is for rows of {plan.d}, got {d}")


def _kind(dtype, bf16, f32):
    if dtype is torch.bfloat16:
        return bf16
    if dtype is torch.float32:
        return f32
    raise ValueError(f"unsupported dtype {dtype}")


def _rope(q, k, positions, plan, q_out, k_out, inverse):
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k are [B, H, T, d]")
    shape, dev, dtype = q.shape, q.device, q.dtype
    B, Hq, T, d = shape
    lib = load()
    fn = _kind(dtype, lib.csa_rope, lib.csa_rope_f32)
    _check_plan(plan, d)
    ps = _position_strides(positions, plan, B, T, dev)
    qs, qos, ks, kos, Hkv = _rows(q, "q", dtype, shape, dev), None, None, None, 0
    if q_out is None:
        q_out = torch.empty(shape, dtype=dtype, device=dev)
    else:
        qos = _rows(q_out, "q_out", dtype, shape, dev, True)
    if k is None:
        k_out = None
    else:
        Hkv = k.shape[1]
        shape = (B, Hkv, T, d)
        ks = _rows(k, "k", dtype, shape, dev)
        if k_out is None:
            k_out = torch.empty(shape, dtype=dtype, device=dev)
        else:
            kos = _rows(k_out, "k_out", dtype, shape, dev, True)
    _check(fn(plan._ref, q.data_ptr(), qs, q_out.data_ptr(), qos, _at(k), ks, _at(k_out), kos, positions.data_ptr(), ps,
              B, Hq, Hkv, T, d, inverse, _raw_stream(dev.index)), "csa_rope")
    return q_out, k_out


def rope(q, k, positions, plan, *, q_out=None, k_out=None, stream=None):
    """Rotary positions on queries and keys.  Returns (q', k').

    q: CUDA [B, Hq, T, d], k: [B, Hkv, T, d] or None, both bf16 or both fp32,
    with any strides whose last one is 1 (for instance slices of one fused
    projection); positions: int32 [axes, B, T] of any strides ([B, T] or [T]
    too for a plan of one axis); plan: a RopeAxes.  q_out, k_out: where the
    results go, the input itself among them (contiguous tensors when None)."""
    if stream is not None or q.device.index is None or q.device.index != _current_device():
        return _there(rope, locals(), q)
    return _rope(q, k, positions, plan, q_out, k_out, 0)


def rope_backward(dq, dk, positions, plan, *, q_out=None, k_out=None, stream=None):
    """Backward pass of rope: the gradients of q and k from the gradients of
    rope's results, rotated by the negative angles.  Arguments as rope."""
    if stream is not None or dq.device.index is None or dq.device.index != _current_device():
        return _there(rope_backward, locals(), dq)
    return _rope(dq, dk, positions, plan, q_out, k_out, 1)


def cache_append(k, v, k_pages, v_pages, block_table, seqlens, *, counts=None, rope=None,
                 positions=None, q=None, q_out=None, stream=None):
    """Writes the rows of new tokens into their pages, the keys rotated if a
    plan is given, and rotates their queries beside.  Returns q' (None without q).

    k, v: CUDA [B, Hkv, T, d] of any strides whose last one is 1, bf16 or
    fp32; row t < counts[b] (int32 [B]; T each when None) becomes token
    seqlens[b] - counts[b] + t of sequence b: seqlens counts the new tokens
    already, as cache_reserve leaves it.  k_pages, v_pages: [P, Hkv, S, d];
    block_table: int32 [B, M].  rope: a RopeAxes; positions as in rope(), or
    None for a token's place in the cache.  q: [B, Hq, T, d], with rope only."""
    if stream is not None or k.device.index is None or k.device.index != _current_device():
        return _there(cache_append, locals(), k)
    if k.dim() != 4 or k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k and v are [B, Hkv, T, d], the pools [P, Hkv, S, d], block_table [B, M]")
    B, Hkv, T, d = k.shape
    P, _, S, _ = k_pages.shape
    M = block_table.shape[1]
    dev, dtype = k.device, k.dtype
    lib = load()
    fn = _kind(dtype, lib.csa_cache_append, lib.csa_cache_append_f32)
    ks = _rows(k, "k", dtype, k.shape, dev)
    vs = _rows(v, "v", dtype, k.shape, dev)
    _need(k_pages, "k_pages", dtype, (P, Hkv, S, d), dev)
    _need(v_pages, "v_pages", dtype, (P, Hkv, S, d), dev)
    _need(block_table, "block_table", torch.int32, (B, M), dev)
    _need(seqlens, "seqlens", torch.int32, (B,), dev)
    if counts is not None:
        _need(counts, "counts", torch.int32, (B,), dev)
    ref = ps = qs = qos = None
    Hq = 0
    if rope is None:
        if q is not None or positions is not None:
            raise ValueError("q and positions go with a rope plan")
        q_out = None
    else:
        _check_plan(rope, d)
        ref = rope._ref
        if positions is not None:
            ps = _position_strides(positions, rope, B, T, dev)
        if q is None:
            q_out = None
        else:
            if q.dim() != 4:
                raise ValueError("q is [B, Hq, T, d]")
            Hq = q.shape[1]
            shape = (B, Hq, T, d)
            qs = _rows(q, "q", dtype, shape, dev)
            if q_out is None:
                q_out = torch.empty(shape, dtype=dtype, device=dev)
            else:
                qos = _rows(q_out, "q_out", dtype, shape, dev, True)
    _check(fn(ref, _at(q), qs, _at(q_out), qos, k.data_ptr(), ks, v.data_ptr(), vs, k_pages.data_ptr(), v_pages.data_ptr(),
              block_table.data_ptr(), seqlens.data_ptr(), _at(counts), _at(positions), ps, B, Hq, Hkv, T, d, P, S, M,
              _raw_stream(dev.index)), "csa_cache_append")
    return q_out


# ------------------------------------------------------------------------ pages
def _books(page_refs, block_table, seqlens):
    dev = page_refs.device
    if page_refs.dim() != 1 or block_table.dim() != 2:
        raise ValueError("page_refs is [P], block_table [B, M]")
    P, (B, M) = page_refs.shape[0], block_table.shape
    _need(page_refs, "page_refs", torch.int32, (P,), dev)
    _need(block_table, "block_table", torch.int32, (B, M), dev)
    _need(seqlens, "seqlens", torch.int32, (B,), dev)
    return dev, P, B, M


def cache_reserve(page_refs, block_table, seqlens, page_size: int, counts, *, shortfall=None, stream=None):
    """Room for counts[b] more tokens of every sequence: takes the missing pages
    (lowest-numbered free ones first), enters them into the table and adds
    counts to seqlens.  Returns shortfall (int32 [1], on the device): 0 if it
    was done, else nothing has changed and it is the number of pages missing
    from the pool, or -1 for a count that does not fit the table.

    page_refs: int32 [P]; block_table: int32 [B, M]; seqlens, counts: int32 [B]."""
    if stream is not None or page_refs.device.index is None or page_refs.device.index != _current_device():
        return _there(cache_reserve, locals(), page_refs)
    dev, P, B, M = _books(page_refs, block_table, seqlens)
    _need(counts, "counts", torch.int32, (B,), dev)
    shortfall = _out(shortfall, "shortfall", torch.int32, (1,), dev)
    _check(load().csa_cache_reserve(page_refs.data_ptr(), block_table.data_ptr(), seqlens.data_ptr(), counts.data_ptr(),
                                    shortfall.data_ptr(), B, P, page_size, M, _raw_stream(dev.index)), "csa_cache_reserve")
    return shortfall


def cache_free(page_refs, block_table, seqlens, page_size: int, rows, *, stream=None):
    """The listed sequences (int32 [R]; -1 is padding) give their pages back:
    their entries become -1, their lengths 0."""
    if stream is not None or page_refs.device.index is None or page_refs.device.index != _current_device():
        return _there(cache_free, locals(), page_refs)
    dev, P, B, M = _books(page_refs, block_table, seqlens)
    R = rows.numel()
    _need(rows, "rows", torch.int32, (R,), dev)
    _check(load().csa_cache_free(page_refs.data_ptr(), block_table.data_ptr(), seqlens.data_ptr(), rows.data_ptr(), R, B, P,
                                 page_size, M, _raw_stream(dev.index)), "csa_cache_free")


def cache_fork(page_refs, block_table, seqlens, page_size: int, parents, children, *, stream=None):
    """children[i] (an empty sequence) becomes a copy of parents[i] (int32 [n]
    both, n <= 4096; a negative entry is padding): full pages are shared, a partly filled
    last page gets a page of its own.  Returns (src, dst, shortfall): the pages
    to copy with cache_copy_pages in every pool (-1 where there is none), and
    shortfall as in cache_reserve."""
    if stream is not None or page_refs.device.index is None or page_refs.device.index != _current_device():
        return _there(cache_fork, locals(), page_refs)
    dev, P, B, M = _books(page_refs, block_table, seqlens)
    n = parents.numel()
    _need(parents, "parents", torch.int32, (n,), dev)
    _need(children, "children", torch.int32, (n,), dev)
    src, dst, shortfall = (torch.empty(size, dtype=torch.int32, device=dev) for size in (n, n, 1))
    _check(load().csa_cache_fork(page_refs.data_ptr(), block_table.data_ptr(), seqlens.data_ptr(), parents.data_ptr(),
                                 children.data_ptr(), n, src.data_ptr(), dst.data_ptr(), shortfall.data_ptr(), B, P,
                                 page_size, M, _raw_stream(dev.index)), "csa_cache_fork")
    return src, dst, shortfall


def cache_compact(page_refs, block_table, seqlens, page_size: int, *, stream=None):
    """Gives the U held pages the numbers 0 .. U - 1.  Returns (src, dst,
    moved): int32 [P // 2] twice and [1]; the pools follow with
    cache_copy_pages(..., src, dst, count=moved) before they are read again."""
    if stream is not None or page_refs.device.index is None or page_refs.device.index != _current_device():
        return _there(cache_compact, locals(), page_refs)
    dev, P, B, M = _books(page_refs, block_table, seqlens)
    half = P // 2
    src, dst, moved = (torch.empty(size, dtype=torch.int32, device=dev) for size in (half, half, 1))
    _check(load().csa_cache_compact(page_refs.data_ptr(), block_table.data_ptr(), seqlens.data_ptr(), src.data_ptr(),
                                    dst.data_ptr(), moved.data_ptr(), B, P, page_size, M, _raw_stream(dev.index)),
           "csa_cache_compact")
    return src, dst, moved


def cache_copy_pages(k_pages, v_pages, src, dst, *, count=None, stream=None):
    """Copies page src[i] onto page dst[i] (int32 [n]; a negative entry is
    padding) for i < min(n, count) in both pools, [P, Hkv, S, d] or, for
    several layers at once, [L, P, Hkv, S, d]; any type.  v_pages may be None;
    count: int32 [1] on the device.  A page that is a dst must not occur in
    another pair."""
    if stream is not None or k_pages.device.index is None or k_pages.device.index != _current_device():
        return _there(cache_copy_pages, locals(), k_pages)
    dev = k_pages.device
    if k_pages.dim() not in (4, 5):
        raise ValueError("the pools are [P, Hkv, S, d] or [L, P, Hkv, S, d]")
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if t is not None:
            _need(t, name, k_pages.dtype, k_pages.shape, dev)
    L = k_pages.shape[0] if k_pages.dim() == 5 else 1
    P, Hkv, S, d = k_pages.shape[-4:]
    n = src.numel()
    _need(src, "src", torch.int32, (n,), dev)
    _need(dst, "dst", torch.int32, (n,), dev)
    if count is not None:
        _need(count, "count", torch.int32, (1,), dev)
    _check(load().csa_cache_copy_pages(_at(k_pages), _at(v_pages), Hkv * S * d * k_pages.element_size(),
                                       L, P, _at(src), _at(dst), n, _at(count), _raw_stream(dev.index)),
           "csa_cache_copy_pages")
