"""Host-side checks of the entry points for 8-bit pools and drafted tokens (no GPU
needed, nothing is launched), and of the host models that the GPU tests use."""
import ctypes
import math

import numpy as np
import pytest
import torch

import continuous_softmax_attention_gb300 as csa
from continuous_softmax_attention_gb300 import _lib as L
from draft_util import DraftBooks, nearest_e4m3, path_of, quantised, scale_of, tree

FAKE, ODD, EIGHT, NULL = ctypes.c_void_p(4096), ctypes.c_void_p(4098), ctypes.c_void_p(4104), None
INV, UNS, ALI, OK = L.CSA_ERR_INVALID_ARG, L.CSA_ERR_UNSUPPORTED, L.CSA_ERR_ALIGNMENT, L.CSA_OK
END = OK if torch.cuda.is_available() else L.CSA_ERR_NO_DEVICE
BF16, F32, E4M3, INT8 = range(4)
IMAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(L.LIB_PATH):
        from continuous_softmax_attention_gb300 import build

        build.build()
    return L.load()


def decode8(lib, *, q=FAKE, k=FAKE, v=FAKE, s=FAKE, k0=NULL, v0=NULL, table=FAKE, lens=FAKE, out=FAKE, lse=NULL, ws=FAKE, nbytes=1 << 40,
            B=2, Hq=8, Hkv=2, P=10, S=16, M=4, d=128, scale=0.1, mode=0, kind=E4M3):
    return lib.csa_decode_paged_q8(q, k, v, s, k0, v0, table, lens, out, lse, ws, nbytes, B, Hq, Hkv, P, S, M, d, scale, mode, kind, None)


def decode_tree(lib, *, q=FAKE, k=FAKE, v=FAKE, s=NULL, k0=NULL, v0=NULL, table=FAKE, lens=FAKE, parents=NULL, counts=NULL, out=FAKE, lse=NULL,
                ws=FAKE, nbytes=1 << 40, B=2, Hq=8, Hkv=2, T=3, P=10, S=16, M=4, d=128, scale=0.1, mode=0, kind=BF16):
    return lib.csa_decode_tree(q, k, v, s, k0, v0, table, lens, parents, counts, out, lse, ws, nbytes, B, Hq, Hkv, T, P, S, M, d, scale, mode,
                               kind, None)


@pytest.mark.parametrize("call", [decode8, decode_tree])
def test_decode_refusals(lib, call):
    tree8 = dict(kind=INT8, s=FAKE) if call is decode_tree else {}
    for kw in (dict(B=-1), dict(Hq=-1), dict(Hkv=0), dict(Hq=7), dict(S=0), dict(M=0), dict(P=-1), dict(d=0), dict(mode=3), dict(mode=-1),
               dict(scale=math.inf), dict(q=NULL), dict(v=NULL), dict(table=NULL), dict(lens=NULL), dict(out=NULL), dict(ws=NULL), dict(mode=2),
               dict(kind=F32), dict(kind=4), dict(kind=-1), {**tree8, "s": NULL, "kind": INT8}):
        assert call(lib, **kw) == INV, kw
    for kw in (dict(d=96), dict(S=12), dict(M=IMAX, B=1), dict(M=2 ** 27, S=16, B=1), dict(B=2 ** 20, M=2 ** 12), dict(P=2 ** 27, S=16),
               {**tree8, "M": 2 ** 28 - 3, "S": 8, "B": 1}):
        assert call(lib, **kw) == UNS, kw
    for kw in (dict(q=ODD), dict(k=ODD), dict(ws=ODD), dict(lens=ODD), dict(table=ODD), dict(mode=2, k0=ODD, v0=FAKE), dict(lse=ODD),
               {**tree8, "s": EIGHT}):
        assert call(lib, **kw) == ALI, kw
    assert call(lib, B=0, q=NULL, k=NULL, v=NULL, s=NULL, table=NULL, lens=NULL, out=NULL, ws=NULL) == OK
    if END != OK:
        assert call(lib) == END and call(lib, **tree8) == END


def test_tree_refusals(lib):
    assert decode_tree(lib, T=-1) == INV and decode_tree(lib, s=FAKE) == INV and decode_tree(lib, T=65) == UNS
    assert decode_tree(lib, parents=ODD) == ALI and decode_tree(lib, counts=ODD) == ALI
    assert decode_tree(lib, T=0, q=NULL, out=NULL, ws=NULL) == OK
    need = lib.csa_decode_tree_workspace_bytes(2, 8, 2, 3, 128)
    assert need > 0 and csa.decode_tree_workspace_bytes(2, 8, 2, 3, 128) == need
    assert decode_tree(lib, nbytes=need - 1) == INV
    for args in ((-1, 8, 2, 3, 128), (1, 7, 2, 3, 128), (1, 8, 0, 3, 128), (1, 8, 2, -1, 128), (1, 8, 2, 65, 128), (1, 8, 2, 3, 96), (2 ** 20, 2 ** 10, 1, 64, 64)):
        assert lib.csa_decode_tree_workspace_bytes(*args) == -1, args
    assert lib.csa_decode_tree_workspace_bytes(0, 8, 2, 3, 128) == 0
    with pytest.raises(csa.CsaError):
        csa.decode_tree_workspace_bytes(1, 8, 2, 65, 128)


def test_append_and_read_refusals(lib):
    def append(*, plan=NULL, q=NULL, qo=NULL, k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, s=FAKE, table=FAKE, lens=FAKE, counts=NULL, pos=NULL, B=2, Hq=0,
               Hkv=2, T=1, d=64, P=4, S=16, M=2, kin=BF16, kind=E4M3):
        return lib.csa_cache_append_q8(plan, q, NULL, qo, NULL, k, NULL, v, NULL, kp, vp, s, table, lens, counts, pos, NULL, B, Hq, Hkv, T, d, P,
                                       S, M, kin, kind, None)

    def read(*, k=FAKE, v=FAKE, s=FAKE, table=FAKE, lens=FAKE, starts=NULL, ko=FAKE, vo=FAKE, B=2, Hkv=2, T=3, d=64, P=4, S=16, M=2, kind=E4M3,
             out=BF16):
        return lib.csa_cache_read(k, v, s, table, lens, starts, ko, NULL, vo, NULL, B, Hkv, T, d, P, S, M, kind, out, None)

    plan = ctypes.byref(csa.RopeAxes(64, (32,))._plan)
    for kw in (dict(k=NULL), dict(v=NULL), dict(kp=NULL), dict(s=NULL), dict(table=NULL), dict(lens=NULL), dict(Hkv=0), dict(S=0), dict(M=0),
               dict(d=0), dict(Hq=2), dict(plan=plan, Hq=2), dict(plan=plan, d=62), dict(T=-1), dict(kin=E4M3), dict(kind=BF16), dict(kind=4)):
        assert append(**kw) == INV, kw
    for kw in (dict(d=300), dict(B=2 ** 16, M=2 ** 16), dict(B=2 ** 16, T=2 ** 16), dict(Hkv=40000)):
        assert append(**kw) == UNS, kw
    for kw in (dict(k=ctypes.c_void_p(4097)), dict(table=ODD), dict(counts=ODD), dict(pos=ODD), dict(s=ctypes.c_void_p(4100)), dict(kin=F32, v=ODD)):
        assert append(**kw) == ALI, kw
    assert append(T=0, k=NULL, v=NULL, kp=NULL, vp=NULL, s=NULL, table=NULL, lens=NULL) == OK
    for kw in (dict(k=NULL), dict(v=NULL), dict(s=NULL), dict(table=NULL), dict(lens=NULL), dict(ko=NULL), dict(vo=NULL), dict(B=-1), dict(Hkv=0),
               dict(T=-1), dict(d=0), dict(kind=4), dict(out=E4M3), dict(kind=BF16), dict(kind=BF16, s=NULL, out=F32), dict(kind=F32, s=NULL)):
        assert read(**kw) == INV, kw
    for kw in (dict(d=257), dict(B=2 ** 16, M=2 ** 16), dict(B=2 ** 12, T=2 ** 18, Hkv=2 ** 4)):
        assert read(**kw) == UNS, kw
    for kw in (dict(ko=ctypes.c_void_p(4097)), dict(out=F32, vo=ODD), dict(s=ctypes.c_void_p(4100)), dict(starts=ODD), dict(lens=ODD)):
        assert read(**kw) == ALI, kw
    assert read(T=0, k=NULL, v=NULL, s=NULL, ko=NULL, vo=NULL, table=NULL, lens=NULL) == OK
    if END != OK:
        assert append() == END and append(plan=plan, Hq=2, q=FAKE, qo=FAKE, kin=F32, kind=INT8) == END
        assert read() == END and read(kind=BF16, s=NULL) == END and read(kind=INT8, out=F32) == END


def test_accept_refusals(lib):
    def accept(*, refs=FAKE, table=FAKE, lens=FAKE, parents=NULL, counts=NULL, last=FAKE, src=FAKE, dst=FAKE, T=3, B=2, P=10, S=16, M=4):
        return lib.csa_cache_accept(refs, table, lens, parents, counts, last, src, dst, T, B, P, S, M, None)

    def copy(*, k=FAKE, v=FAKE, nbytes=64, s=FAKE, sb=8, L=1, P=10, H=2, S=16, src=FAKE, dst=FAKE, groups=1, T=3):
        return lib.csa_cache_copy_rows(k, v, nbytes, s, sb, L, P, H, S, src, dst, groups, T, None)

    for kw in (dict(refs=NULL), dict(table=NULL), dict(lens=NULL), dict(last=NULL), dict(src=NULL), dict(dst=NULL), dict(T=-1), dict(B=-1), dict(S=0)):
        assert accept(**kw) == INV, kw
    assert accept(T=65) == UNS and accept(P=2 ** 28, S=16) == UNS and accept(B=2 ** 16, M=2 ** 16) == UNS
    for kw in (dict(last=ODD), dict(parents=ODD), dict(counts=ODD), dict(src=ODD), dict(refs=ODD)):
        assert accept(**kw) == ALI, kw
    assert accept(B=0, table=NULL, lens=NULL, last=NULL) == OK and accept(T=0, last=NULL, src=NULL, dst=NULL) == OK
    for kw in (dict(k=NULL, v=NULL, s=NULL), dict(src=NULL), dict(dst=NULL), dict(nbytes=-1), dict(sb=-1), dict(L=-1), dict(P=-1), dict(H=-1), dict(S=0),
               dict(groups=-1), dict(T=-1)):
        assert copy(**kw) == INV, kw
    for kw in (dict(T=65), dict(L=65536), dict(H=30000), dict(P=2 ** 28), dict(nbytes=1 << 21)):
        assert copy(**kw) == UNS, kw
    assert copy(src=ODD) == ALI and copy(groups=0) == OK and copy(L=0) == OK and copy(T=0, src=NULL) == OK
    if END != OK:
        assert accept() == END and copy() == END and copy(k=NULL, s=NULL) == END


def test_cpu_tensors_are_refused():
    x, i = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    c, s = torch.zeros(1, 2, 8, 64, dtype=torch.int8), torch.zeros(1, 2, 8, 2)
    for call in (lambda: csa.decode_tree(x, x, x, i[None], i[:1]), lambda: csa.cache_read(c, c, i[None], i[:1], 3, row_scales=s),
                 lambda: csa.cache_append(x, x, c, c, i[None], i[:1], row_scales=s), lambda: csa.cache_accept(i, i[None], i[:1], 16, i[:1], 2),
                 lambda: csa.cache_copy_rows(x, x, i[None], i[None]), lambda: csa.decode_paged(x[:, :, 0], c, c, i[None], i[:1], row_scales=s)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_host_rounding():
    grid = np.array([m * 2.0 ** e for e in range(-9, 6) for m in range(8, 16)] + [m * 2.0 ** -9 for m in range(8)])
    grid = np.unique(grid[grid <= 448])
    y = np.linspace(0, 448, 40001)
    near = nearest_e4m3(y)
    assert np.isin(near, grid).all() and (np.abs(near - y) <= np.abs(grid[:, None] - y).min(0)).all()
    assert (near == torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy())[np.abs(near - y) > 0].all()
    assert scale_of(np.float32([448, 449, 0.0, 2.0 ** -100]), "e4m3").tolist() == [1.0, 2.0, 0.0, 2.0 ** -108]
    c, s = quantised(np.array([[127.0, 63.5, -0.5, 0.4]]), "int8")
    assert s.tolist() == [1.0] and c.tolist() == [[127.0, 64.0, -0.0, 0.0]]


def test_host_model_of_accepted_drafts():
    m = DraftBooks(2, 8, 4, 4)
    assert m.reserve([9, 3]) == 0 and m.table == [[0, 1, 2, -1], [3, -1, -1, -1]]
    parents = [-1, 0, 0, 2, 1]
    assert path_of(parents, 3) == [0, 2, 3] and tree(4, "chain", None) == [-1, 0, 1, 2]
    # sequence 0: 4 tokens, then nodes 0..4 at 4..8; nodes 0, 2, 3 stay
    src, dst = m.accept([parents] * 2, [5, 3], [3, -1], 5)
    assert src == [[-1, 6, 7, -1, -1], [-1] * 5] and dst == [[-1, 5, 6, -1, -1], [-1] * 5]
    assert m.lens == [7, 0] and m.table == [[0, 1, -1, -1], [-1] * 4] and m.refs == [1, 1, 0, 0, 0, 0, 0, 0]
