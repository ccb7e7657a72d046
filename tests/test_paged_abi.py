"""Host-side checks of the paged cache's and the rotary positions' entry points
(no GPU needed, nothing is launched), and of the host model that the GPU tests
compare the page bookkeeping with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import continuous_softmax_attention_gb300 as csa
from continuous_softmax_attention_gb300 import _lib as L
from continuous_softmax_attention_gb300 import _paged
from paged_util import Books, axis_of_pairs, rotated

FAKE, ODD, NULL = ctypes.c_void_p(4096), ctypes.c_void_p(4098), None
INV, UNS, ALI, OK = L.CSA_ERR_INVALID_ARG, L.CSA_ERR_UNSUPPORTED, L.CSA_ERR_ALIGNMENT, L.CSA_OK
END = OK if torch.cuda.is_available() else L.CSA_ERR_NO_DEVICE
IMAX = 2 ** 31 - 1


def ref(plan):
    return ctypes.byref(plan._plan)


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(L.LIB_PATH):
        from continuous_softmax_attention_gb300 import build

        build.build()
    return L.load()


@pytest.fixture
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: valid arguments would launch on fake pointers")


def decode(lib, *, q=FAKE, k=FAKE, v=FAKE, k0=NULL, v0=NULL, table=FAKE, lens=FAKE, out=FAKE, lse=NULL, ws=FAKE, nbytes=1 << 40,
           B=2, Hq=8, Hkv=2, P=10, S=16, M=4, d=128, scale=0.1, mode=0):
    return lib.csa_decode_paged(q, k, v, k0, v0, table, lens, out, lse, ws, nbytes, B, Hq, Hkv, P, S, M, d, scale, mode, None)


def test_decode_paged_refusals(lib):
    need = lib.csa_decode_paged_workspace_bytes(2, 8, 2, 128)
    assert need > 0 and csa.decode_paged_workspace_bytes(2, 8, 2, 128) == need
    for kw in (dict(B=-1), dict(Hq=-1), dict(Hkv=0), dict(Hq=7), dict(S=0), dict(M=0), dict(P=-1), dict(d=0), dict(mode=3), dict(mode=-1),
               dict(scale=math.inf), dict(q=NULL), dict(v=NULL), dict(table=NULL), dict(lens=NULL), dict(out=NULL), dict(ws=NULL),
               dict(nbytes=need - 1), dict(mode=2)):
        assert decode(lib, **kw) == INV, kw
    for kw in (dict(d=96), dict(S=12), dict(M=IMAX, B=1), dict(M=2 ** 27, S=16, B=1), dict(B=2 ** 20, M=2 ** 12), dict(P=2 ** 27, S=16)):
        assert decode(lib, **kw) == UNS, kw
    for kw in (dict(q=ODD), dict(k=ODD), dict(ws=ODD), dict(lens=ODD), dict(table=ODD), dict(mode=2, k0=ODD, v0=FAKE), dict(lse=ODD)):
        assert decode(lib, **kw) == ALI, kw
    assert decode(lib, B=0, q=NULL, k=NULL, v=NULL, table=NULL, lens=NULL, out=NULL, ws=NULL) == OK
    assert lib.csa_decode_paged_workspace_bytes(1, 7, 2, 128) == -1
    assert lib.csa_decode_paged_workspace_bytes(1, 8, 2, 96) == -1
    assert lib.csa_decode_paged_workspace_bytes(-1, 8, 2, 64) == -1
    with pytest.raises(csa.CsaError):
        csa.decode_paged_workspace_bytes(1, 1, 0, 64)


def test_decode_paged_reaches_the_device_check(lib, no_gpu):
    assert decode(lib) == END


def rope(lib, plan, *, q=FAKE, qo=FAKE, k=FAKE, ko=FAKE, pos=FAKE, B=2, Hq=4, Hkv=2, T=3, d=64, f32=False):
    fn = lib.csa_rope_f32 if f32 else lib.csa_rope
    return fn(plan, q, NULL, qo, NULL, k, NULL, ko, NULL, pos, NULL, B, Hq, Hkv, T, d, 0, None)


def test_rope_refusals(lib):
    plan = ref(csa.RopeAxes(64, (10, 22)))
    for kw in (dict(q=NULL), dict(qo=NULL), dict(k=NULL), dict(pos=NULL), dict(B=-1), dict(T=-1), dict(d=0), dict(d=63), dict(Hkv=-1)):
        assert rope(lib, plan, **kw) == INV, kw
    assert rope(lib, NULL) == INV
    assert rope(lib, plan, d=257) == UNS and rope(lib, plan, B=2 ** 20, T=2 ** 12) == UNS and rope(lib, plan, Hq=2 ** 16) == UNS
    assert rope(lib, plan, q=ctypes.c_void_p(4097)) == ALI and rope(lib, plan, f32=True, ko=ODD) == ALI
    assert rope(lib, plan, pos=ODD) == ALI
    assert rope(lib, plan, B=0, q=NULL, qo=NULL, k=NULL, ko=NULL, pos=NULL) == OK
    for field, value in (("pairs", 0), ("pairs", 129), ("axes", 0), ("axes", 9)):
        broken = csa.RopeAxes(64, (10, 22))
        setattr(broken._plan, field, value)
        assert rope(lib, ref(broken)) == INV
    broken = csa.RopeAxes(64, (10, 22))
    broken._plan.axis[5] = 2
    assert rope(lib, ref(broken)) == INV


def test_rope_plan():
    for sections, dealt in (((16, 24, 24), False), ((16, 24, 24), True), ((3, 0, 5, 1), True), ((1,), False)):
        plan = csa.RopeAxes(256, sections, dealt=dealt, base=5e5)
        n = sum(sections)
        assert list(plan._plan.axis)[:n] == axis_of_pairs(sections, dealt)
        for i in range(n):
            turns = 5e5 ** (-i / n) / (2 * math.pi)
            assert abs(plan._plan.turn[i] / 2.0 ** 64 - turns) <= 2.0 ** -51 * turns + 2.0 ** -63
    with pytest.raises(ValueError):
        csa.RopeAxes(64, (1,) * 9)
    with pytest.raises(ValueError):
        csa.RopeAxes(64, (33,))
    with pytest.raises(ValueError):
        csa.RopeAxes(300, (5,))
    with pytest.raises(ValueError):
        csa.RopeAxes(64, (-1, 5))
    for base in (0.0, float("nan"), float("inf")):
        with pytest.raises(csa.CsaError):
            csa.RopeAxes(64, (8,), base=base)
    lib, plan, two = L.load(), _paged._Plan(), (ctypes.c_int * 2)(100, 100)
    assert lib.csa_rope_plan_init(ctypes.byref(plan), two, 2, 1e4, 0) == UNS
    assert lib.csa_rope_plan_init(ctypes.byref(plan), two, 1, 1e4, 4) == INV
    assert lib.csa_rope_plan_init(ctypes.byref(plan), two, 0, 1e4, 0) == INV
    assert lib.csa_rope_plan_init(NULL, two, 1, 1e4, 0) == INV


def test_the_rotation_of_the_inputs_module_is_one_axis():
    from continuous_softmax_attention_gb300.inputs import rope as rope_inputs

    x = torch.randn(1, 2, 9, 32, generator=torch.Generator().manual_seed(0))
    ref = rotated(x, np.arange(9)[None, None], (16,))
    assert np.abs(rope_inputs(x).double().numpy() - ref).max() < 1e-5


def append(lib, *, plan=NULL, q=NULL, qo=NULL, k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE, counts=NULL, pos=NULL, B=2, Hq=0,
           Hkv=2, T=1, d=64, P=4, S=16, M=2):
    return lib.csa_cache_append(plan, q, NULL, qo, NULL, k, NULL, v, NULL, kp, vp, table, lens, counts, pos, NULL, B, Hq, Hkv, T, d, P, S, M,
                                None)


def test_append_refusals(lib):
    plan = ref(csa.RopeAxes(64, (32,)))
    for kw in (dict(k=NULL), dict(v=NULL), dict(kp=NULL), dict(table=NULL), dict(lens=NULL), dict(Hkv=0), dict(S=0), dict(M=0), dict(d=0),
               dict(Hq=2), dict(plan=plan, Hq=2), dict(plan=plan, d=62), dict(T=-1)):
        assert append(lib, **kw) == INV, kw
    for kw in (dict(d=300), dict(B=2 ** 16, M=2 ** 16), dict(B=2 ** 16, T=2 ** 16), dict(Hkv=40000)):
        assert append(lib, **kw) == UNS, kw
    for kw in (dict(k=ctypes.c_void_p(4097)), dict(table=ODD), dict(counts=ODD), dict(pos=ODD)):
        assert append(lib, **kw) == ALI, kw
    assert append(lib, T=0, k=NULL, v=NULL, kp=NULL, vp=NULL, table=NULL, lens=NULL) == OK


def test_page_calls_refuse(lib):
    def reserve(refs=FAKE, table=FAKE, lens=FAKE, counts=FAKE, short=FAKE, B=2, P=10, S=16, M=4):
        return lib.csa_cache_reserve(refs, table, lens, counts, short, B, P, S, M, None)

    def free(rows=FAKE, R=1, refs=FAKE, B=2, P=10, S=16, M=4):
        return lib.csa_cache_free(refs, FAKE, FAKE, rows, R, B, P, S, M, None)

    def fork(parents=FAKE, n=1, src=FAKE, short=FAKE, B=2, M=4):
        return lib.csa_cache_fork(FAKE, FAKE, FAKE, parents, FAKE, n, src, FAKE, short, B, 10, 16, M, None)

    def compact(src=FAKE, moved=FAKE, P=10):
        return lib.csa_cache_compact(FAKE, FAKE, FAKE, src, FAKE, moved, 2, P, 16, 4, None)

    def copy(k=FAKE, nbytes=64, layers=1, P=10, src=FAKE, dst=FAKE, n=1, count=NULL):
        return lib.csa_cache_copy_pages(k, NULL, nbytes, layers, P, src, dst, n, count, None)

    for kw in (dict(refs=NULL), dict(table=NULL), dict(lens=NULL), dict(counts=NULL), dict(short=NULL), dict(S=0), dict(M=0), dict(B=-1), dict(P=-1)):
        assert reserve(**kw) == INV, kw
    assert reserve(B=2 ** 16, M=2 ** 16) == UNS and reserve(S=2 ** 30) == UNS
    assert reserve(refs=ODD) == ALI and reserve(counts=ODD) == ALI
    assert free(rows=NULL) == INV and free(R=-1) == INV and free(rows=ODD) == ALI and free(refs=NULL) == INV and free(R=0) == OK
    assert fork(parents=NULL) == INV and fork(n=-1) == INV and fork(src=NULL) == INV and fork(short=NULL) == INV
    assert fork(src=ODD) == ALI and fork(n=4097) == UNS
    assert compact(moved=NULL) == INV and compact(src=NULL) == INV and compact(src=ODD) == ALI
    assert copy(k=NULL) == INV and copy(src=NULL) == INV and copy(n=-1) == INV and copy(nbytes=-1) == INV and copy(layers=-1) == INV
    assert copy(src=ODD) == ALI and copy(n=0) == OK and copy(layers=0) == OK
    assert copy(nbytes=1 << 40, layers=1 << 20, P=1 << 20) == UNS


def test_valid_calls_reach_the_device_check(lib, no_gpu):
    plan = ref(csa.RopeAxes(64, (32,)))
    assert rope(lib, plan) == END and append(lib) == END and append(lib, plan=plan, Hq=2, q=FAKE, qo=FAKE) == END
    assert lib.csa_cache_reserve(*[FAKE] * 5, 2, 10, 16, 4, None) == END
    assert lib.csa_cache_free(FAKE, FAKE, FAKE, FAKE, 1, 2, 10, 16, 4, None) == END
    assert lib.csa_cache_compact(*[FAKE] * 6, 2, 10, 16, 4, None) == END


def test_cpu_tensors_are_refused():
    x, i = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    plan = csa.RopeAxes(64, (32,))
    for call in (lambda: csa.rope(x, x, i[:3], plan), lambda: csa.cache_append(x, x, x, x, i[None], i[:1]),
                 lambda: csa.cache_free(i, i[None], i[:1], 16, i), lambda: csa.cache_copy_pages(x, x, i, i),
                 lambda: csa.decode_paged(x[:, :, 0], x, x, i[None], i[:1])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_missing_module_is_reported(monkeypatch):
    monkeypatch.setattr(_paged, "_native", _paged._Unloaded())
    monkeypatch.setitem(__import__("sys").modules, "continuous_softmax_attention_gb300._csa_torch", None)
    monkeypatch.delattr(csa, "_csa_torch", raising=False)
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="build it"):
        csa.rope(x, None, torch.zeros(1, 1, 3, dtype=torch.int32), csa.RopeAxes(64, (32,)))


def test_host_model_of_the_pages():
    m = Books(4, 8, 4, 4)
    assert m.reserve([5, 4, 0, 0]) == 0 and m.table[:2] == [[0, 1, -1, -1], [2, -1, -1, -1]]
    assert m.fork([0, 1], [2, 3]) == ([1, -1], [3, -1], 0)
    assert m.refs == [2, 1, 2, 1, 0, 0, 0, 0] and m.table[2] == [0, 3, -1, -1]
    m.free([0, 1, 0])
    assert m.refs == [1, 0, 1, 1, 0, 0, 0, 0] and m.lens == [0, 0, 5, 4]
    assert m.compact() == ([3], [1]) and m.table[2:] == [[0, 1, -1, -1], [2, -1, -1, -1]]
    assert m.reserve([0, 0, 12, 0]) == -1 and m.reserve([16, 16, 0, 0]) == 3
