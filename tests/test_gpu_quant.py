"""Rows quantised into 8-bit pages (csa_cache_append_q8) and rows read back
(csa_cache_read), against the host's rounding of the same values."""
import numpy as np
import pytest
import torch

from continuous_softmax_attention_gb300 import CsaError, RopeAxes, cache_append, cache_read, device_status, rope
from draft_util import KINDS, half_step, quantised, random_pools, values
from paged_util import HALF_STEP, pages_of, rope_bound, rotated, scattered

pytestmark = pytest.mark.gpu

EIGHT = pytest.mark.parametrize("kind", ["e4m3", "int8"])
INT = dict(dtype=torch.int32, device="cuda")


def bits(x):
    return x.cpu().view(torch.uint8).numpy()


def case(B, Hq, Hkv, T, d, S, kind, seed, dtype=torch.bfloat16, counts=None, past=20):
    g = torch.Generator().manual_seed(seed)
    r = np.random.default_rng(seed)
    counts = [int(r.integers(0, T + 1)) for _ in range(B)] if counts is None else counts
    lens = [int(r.integers(0, past + 1)) + c for c in counts]
    P = sum(pages_of(n, S) for n in lens) + 3
    k, v, scales = random_pools(P, Hkv, S, d, kind, g)
    x = torch.randn(B, T, Hq + 2 * Hkv, d, generator=g).to(dtype)
    return dict(x=x, k_pages=k, v_pages=v, scales=scales, table=scattered(lens, S, P, seed), lens=lens, counts=counts, Hq=Hq, Hkv=Hkv, S=S)


def on_gpu(c):
    x = c["x"].cuda()
    Hq, Hkv = c["Hq"], c["Hkv"]
    return dict(q=x[:, :, :Hq].transpose(1, 2), k=x[:, :, Hq:Hq + Hkv].transpose(1, 2), v=x[:, :, Hq + Hkv:].transpose(1, 2),
                k_pages=c["k_pages"].cuda(), v_pages=c["v_pages"].cuda(), scales=c["scales"].cuda(),
                table=torch.as_tensor(c["table"]).cuda(), lens=torch.tensor(c["lens"], **INT), counts=torch.tensor(c["counts"], **INT))


def append(u, **kw):
    return cache_append(u["k"], u["v"], u["k_pages"], u["v_pages"], u["table"], u["lens"], row_scales=u["scales"], counts=u["counts"], **kw)


def new_rows(c):
    """(b, t, page, slot) of every new row."""
    S = c["S"]
    return [(b, t, c["table"][b][(n - m + t) // S], (n - m + t) % S) for b, (n, m) in enumerate(zip(c["lens"], c["counts"])) for t in range(m)]


def check_pools(c, u, keys, vals, kind, exact):
    """Every new row is the rounding of its values (bit for bit where they are exact), every other byte as it was."""
    k, v, s = bits(u["k_pages"]), bits(u["v_pages"]), u["scales"].cpu().numpy()
    k0, v0, s0 = bits(c["k_pages"]).copy(), bits(c["v_pages"]).copy(), c["scales"].numpy().copy()
    as_values = lambda raw: torch.from_numpy(raw.copy()).view(KINDS[kind]).float().numpy().astype(np.float64)  # noqa: E731
    for b, t, page, slot in new_rows(c):
        for raw, raw0, x, i, err in ((k, k0, keys[0], 0, keys[1]), (v, v0, vals, 1, None)):
            want, scale = quantised(x[b, :, t], kind)
            got, gs = as_values(raw[page, :, slot]), s[page, :, slot, i]
            if err is None or exact:
                assert (gs == scale).all() and (got == want).all(), (b, t, i)
            else:  # turned in fp32: off by err before the rounding
                e = err[b, :, t]
                assert (np.abs(got * gs[:, None] - x[b, :, t]) <= half_step(np.abs(x[b, :, t]) + e, gs, kind) + e).all()
                near = np.abs(gs / scale - 1) <= 2.0 ** -20
                if kind == "e4m3":  # where the largest value is within err of a border, the next power of two may be taken
                    near |= (np.abs(np.log2(gs / scale)) == 1) & (np.abs(np.abs(x[b, :, t]).max(-1) / np.minimum(gs, scale) - 448) < 0.01)
                assert near.all()
            raw0[page, :, slot] = raw[page, :, slot]
            s0[page, :, slot, i] = gs
    assert (k == k0).all() and (v == v0).all() and (s.view(np.int32) == s0.view(np.int32)).all()


@EIGHT
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,S", [(128, 16), (64, 24), (256, 8), (80, 5), (33, 16), (1, 3), (250, 1)])
def test_rows_are_rounded_to_nearest(kind, dtype, d, S):
    c = case(3, 0, 2, 9, d, S, kind, seed=d + S, dtype=dtype, counts=[9, 0, 4])
    c["x"][0, 0] = torch.linspace(-1, 1, d).to(dtype)        # ties of int8, and equal magnitudes
    c["x"][0, 1] = (torch.arange(d) % 29 / 16 * 256 / 2).to(dtype)  # ties of e4m3
    c["x"][0, 2] = 0
    c["x"][0, 3] = 2.0 ** -101
    c["x"][0, 4] *= 2.0 ** -96
    c["x"][0, 5] *= 2.0 ** 120
    c["x"][0, 6, :, :1] = 448.0
    c["x"][0, 7, :, :1] = 450.0
    u = on_gpu(c)
    append(u)
    torch.cuda.synchronize()
    x = c["x"].double().numpy().transpose(0, 2, 1, 3)
    check_pools(c, u, (x[:, :2], None), x[:, 2:], kind, True)
    assert device_status() == 0


@EIGHT
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,sections,kw", [(128, (16, 24, 24), {}), (128, (20, 12), dict(adjacent=True)), (64, (8, 8), dict(dealt=True)), (96, (48,), {}),
                                           (256, (100, 28), dict(adjacent=True, dealt=True)), (50, (7, 11), {}), (256, (128,), {}), (250, (101, 2), {})])
def test_keys_turn_and_queries_beside(kind, dtype, d, sections, kw):
    c = case(3, 4, 2, 11, d, 16, kind, seed=d, dtype=dtype, past=3000)
    u = on_gpu(c)
    plan = RopeAxes(d, sections, **kw)
    pos = torch.randint(-5, 100000, (len(sections), 3, 11), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    q = append(u, rope=plan, positions=pos.cuda(), q=u["q"])
    x = c["x"].transpose(1, 2)
    rq, rk = (rotated(t, pos, sections, **kw) for t in (x[:, :4], x[:, 4:6]))
    assert (np.abs(q.double().cpu().numpy() - rq) <= rope_bound(x[:, :4], rq)).all()
    err = np.full(rk.shape, 2 * (4 + 2) * 2.0 ** -24 * x[:, 4:6].float().abs().max().item())
    check_pools(c, u, (rk, err), x[:, 6:].double().numpy(), kind, False)
    # the same queries as the call for pools of the inputs' type gives
    assert torch.equal(q, rope(u["q"], None, pos.cuda(), plan)[0])
    assert device_status() == 0


@EIGHT
def test_positions_default_to_the_place_in_the_cache(kind):
    c = case(4, 2, 1, 5, 64, 8, kind, seed=3)
    u, w = on_gpu(c), on_gpu(c)
    plan = RopeAxes(64, (20, 12))
    at = torch.tensor([[n - m + t for t in range(5)] for n, m in zip(c["lens"], c["counts"])], **INT)
    a, b = append(u, rope=plan, q=u["q"]), append(w, rope=plan, q=w["q"], positions=at.expand(2, 4, 5))
    assert torch.equal(a, b) and (bits(u["k_pages"]) == bits(w["k_pages"])).all() and torch.equal(u["scales"], w["scales"])


@EIGHT
def test_rows_of_any_alignment(kind):
    """Slices that begin off 16 bytes take the path of single elements: the same codes."""
    c = case(2, 0, 3, 7, 64, 16, kind, seed=4)
    u, w = on_gpu(c), on_gpu(c)
    wide = torch.zeros(2, 3, 7, 67, dtype=torch.bfloat16, device="cuda")
    wide[..., 1:65] = w["k"]
    w["k"] = wide[..., 1:65]
    append(u)
    append(w)
    assert (bits(u["k_pages"]) == bits(w["k_pages"])).all() and (bits(u["v_pages"]) == bits(w["v_pages"])).all()
    assert torch.equal(u["scales"], w["scales"])


@EIGHT
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_rows_that_are_not_finite_read_as_nan(kind, bad):
    c = case(1, 0, 2, 3, 128, 16, kind, seed=5, counts=[3])
    c["x"][0, 1, 1, 77] = bad
    u = on_gpu(c)
    append(u)
    k, v = cache_read(u["k_pages"], u["v_pages"], u["table"], u["lens"], 3, starts=u["lens"] - 3, row_scales=u["scales"])
    assert torch.isnan(k[0, 1, 1]).all() and torch.isfinite(k[0, 0]).all() and torch.isfinite(k[0, 1, ::2]).all() and torch.isfinite(v).all()


@EIGHT
def test_bad_lengths_and_pages_are_not_written(kind):
    c = case(4, 0, 1, 6, 64, 8, kind, seed=6, counts=[6, 6, 6, 6], past=10)
    u = on_gpu(c)
    u["counts"][0], u["lens"][1] = 7, 5  # more than T; fewer than the count
    n = c["lens"][2]
    u["table"][2, (n - 1) // 8] = 10 ** 6
    u["lens"][3] = u["table"].shape[1] * 8 + 1
    append(u)
    torch.cuda.synchronize()
    assert device_status() == -1 and device_status() == 0
    lost = {(2, t) for t in range(6) if (n - 6 + t) // 8 == (n - 1) // 8}
    k0 = bits(c["k_pages"]).copy()
    k = bits(u["k_pages"])
    for b, t, page, slot in new_rows(c):
        if b == 2 and (b, t) not in lost:
            assert (k[page, :, slot] != k0[page, :, slot]).any()
            k0[page, :, slot] = k[page, :, slot]
    assert (k == k0).all()


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3", "int8"])
@pytest.mark.parametrize("d,S", [(128, 16), (64, 24), (256, 8), (80, 7), (33, 16), (1, 3), (8, 4)])
def test_read_in_order(kind, d, S):
    g = torch.Generator().manual_seed(d)
    lens, starts, T = [0, 1, 50, 37, S, 3 * S], [0, 0, 13, 37, 0, S], 41
    P = sum(pages_of(n, S) for n in lens) + 2
    k, v, scales = random_pools(P, 3, S, d, "bf16" if kind == "f32" else kind, g, spread=20.0)
    if kind == "f32":
        k, v = torch.randn(P, 3, S, d, generator=g), torch.randn(P, 3, S, d, generator=g)
    table = scattered(lens, S, P, d)
    vk, vv = values(k, v, scales)
    kw = dict(row_scales=scales.cuda()) if scales is not None else {}
    args = (k.cuda(), v.cuda(), torch.as_tensor(table).cuda(), torch.tensor(lens, **INT), T)
    for dtype in (None, torch.float32) if scales is not None else (None,):
        ok, ov = cache_read(*args, starts=torch.tensor(starts, **INT), dtype=dtype, **kw)
        want_type = dtype or (torch.bfloat16 if scales is not None else k.dtype)
        for got, val in ((ok, vk), (ov, vv)):
            assert got.dtype is want_type and got.shape == (6, 3, T, d)
            want = torch.zeros(6, 3, T, d, dtype=torch.float64)
            for b, (n, s0) in enumerate(zip(lens, starts)):
                for t in range(min(T, n - s0)):
                    want[b, :, t] = val[table[b][(s0 + t) // S], :, (s0 + t) % S]
            got = got.cpu()
            if scales is None:
                assert torch.equal(got.double(), want)
            elif dtype is torch.float32:  # a code of 8 bits times a scale of 24, rounded once
                assert torch.equal(got, want.float())
            else:  # fp32, then bf16: a second rounding can move a tie
                assert ((got.double() - want).abs() <= HALF_STEP[torch.bfloat16] * want.abs() * (1 + 2.0 ** -15)).all()
    a, _ = cache_read(*args, **kw)
    z, _ = cache_read(*args, starts=torch.zeros(6, **INT), **kw)
    assert torch.equal(a, z) and device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_read_into_slices(kind):
    g = torch.Generator().manual_seed(7)
    k, v, scales = random_pools(9, 2, 16, 64, kind, g)
    table = scattered([40, 70], 16, 9, 1)
    kw = dict(row_scales=scales.cuda()) if scales is not None else {}
    args = (k.cuda(), v.cuda(), torch.as_tensor(table).cuda(), torch.tensor([40, 70], **INT), 30)
    rk, rv = cache_read(*args, **kw)
    for lead in (0, 8, 1):  # aligned and not
        buf = torch.full((2, 30, 2, 2 * 64 + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        ko, vo = (buf[..., lead + i * 64:lead + i * 64 + 64].transpose(1, 2) for i in range(2))
        before = ko._version
        ok, ov = cache_read(*args, k_out=ko, v_out=vo, **kw)
        assert torch.equal(ok, rk) and torch.equal(ov, rv) and ok.data_ptr() == ko.data_ptr() and buf._version > before
        assert (buf[..., :lead] == 7).all() and (buf[..., lead + 128:] == 7).all()


@pytest.mark.parametrize("kind", ["f32", "int8"])
def test_read_shows_bad_lengths_and_pages(kind):
    k, v, scales = random_pools(8, 1, 4, 32, "int8" if kind == "int8" else "bf16", torch.Generator().manual_seed(8))
    if kind == "f32":
        k, v = k.float(), v.float()
    table = torch.arange(8, **INT).view(4, 2).clone()
    table[3, 1] = -1
    kw = dict(row_scales=scales.cuda()) if scales is not None else {}
    ok, ov = cache_read(k.cuda(), v.cuda(), table, torch.tensor([8, 9, 5, 8], **INT), 8, starts=torch.tensor([-1, 0, 6, 0], **INT), **kw)
    assert torch.isnan(ok[:3]).all() and torch.isnan(ov[:3]).all()
    assert torch.isfinite(ok[3, :, :4]).all() and torch.isnan(ok[3, :, 4:]).all()
    assert device_status() == -1 and device_status() == 0


def test_arguments_are_checked():
    c = case(2, 2, 1, 3, 64, 8, "int8", seed=9)
    u = on_gpu(c)
    ok = (u["k"], u["v"], u["k_pages"], u["v_pages"], u["table"], u["lens"])
    for args, kw in (((ok), {}),                                                             # no scales
                     ((*ok[:2], u["k_pages"].to(torch.bfloat16), u["v_pages"].to(torch.bfloat16), *ok[4:]), dict(row_scales=u["scales"])),
                     ((*ok[:3], u["v_pages"].float().to(torch.float8_e4m3fn), *ok[4:]), dict(row_scales=u["scales"])),
                     (ok, dict(row_scales=u["scales"][..., :1])), (ok, dict(row_scales=u["scales"].double())),
                     (ok, dict(row_scales=u["scales"].cpu())), (ok, dict(row_scales=u["scales"], q=u["q"]))):
        with pytest.raises(ValueError):
            cache_append(*args, **kw)
    for args, kw in (((*ok[2:], 4), {}), ((*ok[2:], -1), dict(row_scales=u["scales"])), ((*ok[2:], 4), dict(row_scales=u["scales"], dtype=torch.float16)),
                     ((*ok[2:], 4), dict(row_scales=u["scales"], starts=u["lens"].long())),
                     ((*ok[2:], 4), dict(row_scales=u["scales"], k_out=torch.zeros(2, 1, 4, 64, device="cuda")))):
        with pytest.raises(ValueError):
            cache_read(*args, **kw)
    with pytest.raises(CsaError):  # more columns than a row may have
        big = torch.zeros(1, 1, 8, 300, dtype=torch.int8, device="cuda")
        cache_read(big, big, torch.zeros(1, 1, **INT), torch.ones(1, **INT), 1, row_scales=torch.ones(1, 1, 8, 2, device="cuda"))
    before = u["k_pages"]._version, u["scales"]._version
    cache_append(*ok, row_scales=u["scales"], counts=u["counts"])
    assert u["k_pages"]._version > before[0] and u["scales"]._version > before[1]
    empty = cache_read(*ok[2:], 0, row_scales=u["scales"])
    assert empty[0].shape == (2, 1, 0, 64)


@EIGHT
def test_in_a_graph_and_on_a_given_stream(kind):
    c = case(3, 2, 2, 4, 64, 8, kind, seed=10, counts=[4, 4, 4])
    u = on_gpu(c)
    plan = RopeAxes(64, (32,))
    q = append(u, rope=plan, q=u["q"])
    want = q.clone(), bits(u["k_pages"]).copy(), u["scales"].clone()
    k, v = cache_read(u["k_pages"], u["v_pages"], u["table"], u["lens"], 9, row_scales=u["scales"])
    s = torch.cuda.Stream()
    w = on_gpu(c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        gq = append(w, rope=plan, q=w["q"])
        gk, gv = cache_read(w["k_pages"], w["v_pages"], w["table"], w["lens"], 9, row_scales=w["scales"])
    for _ in range(2):
        w["k_pages"].view(torch.uint8).fill_(0)
        w["k_pages"].copy_(c["k_pages"])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(gq, want[0]) and (bits(w["k_pages"]) == want[1]).all() and torch.equal(w["scales"], want[2])
        assert torch.equal(gk, k) and torch.equal(gv, v)
    w = on_gpu(c)
    torch.cuda.synchronize()
    append(w, rope=plan, q=w["q"], stream=s)
    k2, _ = cache_read(w["k_pages"], w["v_pages"], w["table"], w["lens"], 9, row_scales=w["scales"], stream=s)
    s.synchronize()
    assert torch.equal(k2, k)


def test_rows_far_into_a_pool():
    """A pool of more than 2^32 bytes: codes and scales go to their own rows."""
    P, H, S, d = 20000, 8, 128, 256  # 5.2 GB a pool
    k = torch.zeros(P, H, S, d, dtype=torch.int8, device="cuda")
    scales = torch.zeros(P, H, S, 2, device="cuda")
    table = torch.tensor([[P - 1, 3]], **INT)
    x = torch.randn(1, H, 130, d, generator=torch.Generator().manual_seed(11)).to(torch.bfloat16).cuda()
    n = torch.tensor([130], **INT)
    cache_append(x, x, k, k, table, n, row_scales=scales)
    out, _ = cache_read(k, k, table, n, 130, row_scales=scales, dtype=torch.float32)
    want, s = x.double().cpu().numpy()[0], scales[P - 1].cpu().numpy()[..., 0]
    got = out.double().cpu().numpy()[0]
    assert (np.abs(got[:, :S] - want[:, :S]) <= half_step(want[:, :S], s, "int8")).all()
    assert (np.abs(got[:, S:] - want[:, S:]) <= half_step(want[:, S:], scales[3].cpu().numpy()[:, :2, 0], "int8")).all()
    assert (k[P - 1].float().abs().sum(-1) > 0).all() and (k[1:3] == 0).all() and (k[P - 2] == 0).all()
