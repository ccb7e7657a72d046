"""Rotary positions with several axes (csa_rope, its backward pass, and the
append that rotates keys into pages) against 64-bit rotations."""
import numpy as np
import pytest
import torch

from continuous_softmax_attention_gb300 import CsaError, RopeAxes, cache_append, device_status, rope, rope_backward
from paged_util import pages_of, rope_bound, rotated, scattered

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def tensors(B, T, Hq, Hkv, d, dtype, seed, fused):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, Hq + 2 * Hkv, d, generator=g).to(DT[dtype]).cuda()
    q, k, v = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2), x[:, :, Hq + Hkv:].transpose(1, 2)
    return (q, k, v) if fused else tuple(t.contiguous() for t in (q, k, v))


def draw_positions(A, B, T, far, seed):
    return torch.randint(-far // 2, far, (A, B, T), generator=torch.Generator().manual_seed(seed), dtype=torch.int64).int().cuda()


def same(got, x, ref):
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= rope_bound(x, ref)).all(), float((err / rope_bound(x, ref)).max())


SPECS = [  # d, sections, adjacent, dealt
    (128, (16, 24, 24), False, False), (128, (64,), False, False), (128, (64,), True, False), (64, (10, 11, 11), True, True),
    (256, (30, 49, 49), False, True), (128, (8, 16), False, False), (96, (17, 7), True, False), (80, (40,), False, False),
    (2, (1,), False, False), (7, (2, 1), True, True), (63, (0, 5, 9), False, True), (130, (1, 2, 3, 4, 5, 6, 7, 8), False, True)]


@pytest.mark.parametrize("spec", SPECS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fused", [False, True])
def test_forward_and_backward(spec, dtype, fused):
    d, sections, adjacent, dealt = spec
    B, T, Hq, Hkv = 2, 19, 5, 3
    plan = RopeAxes(d, sections, adjacent=adjacent, dealt=dealt)
    q, k, _ = tensors(B, T, Hq, Hkv, d, dtype, d, fused)
    pos = draw_positions(len(sections), B, T, 5000, 1)
    kw = dict(adjacent=adjacent, dealt=dealt)
    for fn, inverse in ((rope, False), (rope_backward, True)):
        qo, ko = fn(q, k, pos, plan)
        assert qo.is_contiguous() and ko.is_contiguous()
        same(qo, q, rotated(q, pos, sections, inverse=inverse, **kw))
        same(ko, k, rotated(k, pos, sections, inverse=inverse, **kw))


@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (64, 1, 32, 8), (1, 700, 32, 8), (3, 33, 1, 4), (2, 5, 0, 2)])
def test_shapes(B, T, Hq, Hkv):
    plan = RopeAxes(128, (16, 24, 24))
    q, k, _ = tensors(B, T, Hq, Hkv, 128, "bf16", T, True)
    pos = draw_positions(3, B, T, 1 << 20, 2)
    qo, ko = rope(q, k, pos, plan)
    if Hq:
        same(qo, q, rotated(q, pos, (16, 24, 24)))
    same(ko, k, rotated(k, pos, (16, 24, 24)))


def test_far_and_negative_positions():
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 12345679], dtype=torch.int32).cuda()
    for base in (10000.0, 500000.0, 1e7):
        plan = RopeAxes(64, (32,), base=base)
        q, _, _ = tensors(1, 8, 2, 1, 64, "f32", 3, False)
        qo, none = rope(q, None, pos, plan)
        assert none is None
        same(qo, q, rotated(q, pos[None, None].cpu(), (32,), base=base))


def test_gradient_against_differences():
    # L = sum(dout * rope(x)): dL/dx against central differences; L is linear in x, so a wide step is exact
    plan = RopeAxes(16, (3, 4), dealt=True)
    x, _, _ = tensors(1, 3, 2, 1, 16, "f32", 4, False)
    pos = draw_positions(2, 1, 3, 100, 5)
    dout = torch.randn(x.shape, generator=torch.Generator().manual_seed(6)).cuda()
    dx, _ = rope_backward(dout, None, pos, plan)
    for i in range(0, x.numel(), 5):
        e = torch.zeros_like(x).flatten()
        e[i] = 4.0
        up, down = (rope(x + s * e.view_as(x), None, pos, plan)[0].double() for s in (1, -1))
        slope = ((up - down) * dout.double()).sum().item() / 8.0
        # two outputs rounded to fp32 at magnitude <= 10, over 16 entries
        assert abs(slope - dx.flatten()[i].item()) <= 2.0 ** -24 * 10 * 16 * dout.abs().max().item()


def test_inverse_undoes_and_zero_positions_copy():
    plan = RopeAxes(128, (20, 20), adjacent=True)
    q, k, _ = tensors(2, 9, 4, 2, 128, "f32", 7, True)
    pos = draw_positions(2, 2, 9, 10 ** 6, 8)
    back, _ = rope_backward(*rope(q, k, pos, plan), pos, plan)
    assert (back - q).abs().max().item() <= 24 * 2.0 ** -24 * q.abs().max().item()
    qo, ko = rope(q, k, torch.zeros_like(pos), plan)
    assert torch.equal(qo, q) and torch.equal(ko, k)
    assert torch.equal(rope(q, k, pos, plan)[0][..., 80:], q[..., 80:])


def test_in_place_and_strided_outputs():
    plan = RopeAxes(128, (16, 24, 24))
    q, k, v = tensors(2, 33, 6, 2, 128, "bf16", 9, True)
    pos = draw_positions(3, 2, 33, 1 << 18, 10)
    qo, ko = rope(q, k, pos, plan)
    whole = torch.zeros(2, 33, 10, 128, dtype=torch.bfloat16, device="cuda")  # another fused buffer
    qv, kv = whole[:, :, :6].transpose(1, 2), whole[:, :, 6:8].transpose(1, 2)
    a, b = rope(q, k, pos, plan, q_out=qv, k_out=kv)
    assert a is qv and torch.equal(qv, qo) and torch.equal(kv, ko) and not whole[:, :, 8:].any()
    before = v.clone()
    rope(q, k, pos, plan, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, before)


def test_broadcast_positions_and_odd_alignment():
    plan = RopeAxes(64, (16, 16))
    base = torch.randn(2 * 4 * 5 * 64 + 1, generator=torch.Generator().manual_seed(11)).to(torch.bfloat16).cuda()
    q = base[1:].view(2, 4, 5, 64)  # 2-byte aligned only
    pos = draw_positions(2, 1, 5, 1000, 12).expand(2, 2, 5)
    qo, _ = rope(q, None, pos, plan)
    same(qo, q, rotated(q, pos, (16, 16)))
    qb = q[:1].expand(2, 4, 5, 64)  # one input for both batch entries
    qo, _ = rope(qb, None, pos, plan)
    same(qo, q, rotated(qb, pos, (16, 16)))


def test_long_offsets():
    # rows beyond 2^31 elements of one tensor
    T, H = 2 ** 24 + 3, 2
    q = torch.zeros(1, H, T, 128, dtype=torch.bfloat16, device="cuda")
    q[0, 1, -2:] = torch.randn(2, 128, device="cuda").to(torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    tail = q[:, :, -2:].clone()
    plan = RopeAxes(128, (64,))
    rope(q, None, pos, plan, q_out=q)
    same(q[:, :, -2:], tail, rotated(tail, pos[None, None, -2:].cpu(), (64,)))


# ------------------------------------------------------------------------------ append
def pools(P, Hkv, S, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(P, Hkv, S, d, generator=g).to(DT[dtype]).cuda() for _ in range(2)]


def expected(k, v, kp, vp, table, lens, counts, S, turn):
    """Pools after the append, in 64 bits, one row at a time."""
    kr, vr = turn(k), v.double().cpu().numpy()
    ke, ve = kp.double().cpu().numpy().copy(), vp.double().cpu().numpy().copy()
    for b, (n, c) in enumerate(zip(lens, counts)):
        for t in range(c):
            page, place = table[b, (n - c + t) // S], (n - c + t) % S
            ke[page, :, place], ve[page, :, place] = kr[b, :, t], vr[b, :, t]
    return ke, ve


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S,d,spec", [(16, 128, (16, 24, 24)), (8, 64, (32,)), (5, 40, (6, 7)), (24, 256, (60, 60))])
@pytest.mark.parametrize("T", [1, 37])
def test_append(dtype, S, d, spec, T):
    counts = [T, 0, T, min(T, 3)]
    lens = [T, 0, 100 + T, 50]
    Hq, Hkv = 6, 2
    table = scattered(lens, S, sum(pages_of(n, S) for n in lens) + 2, 1)
    kp, vp = pools(sum(pages_of(n, S) for n in lens) + 2, Hkv, S, d, dtype, 2)
    q, k, v = tensors(4, T, Hq, Hkv, d, dtype, 3, True)
    pos = draw_positions(len(spec), 4, T, 9000, 4)
    plan = RopeAxes(d, spec)
    ke, ve = expected(k, v, kp, vp, table, lens, counts, S, lambda x: rotated(x, pos, spec))
    ints = dict(dtype=torch.int32, device="cuda")
    qo = cache_append(k, v, kp, vp, torch.as_tensor(table).cuda(), torch.tensor(lens, **ints),
                      counts=torch.tensor(counts, **ints), rope=plan, positions=pos, q=q)
    torch.cuda.synchronize()
    same(qo, q, rotated(q, pos, spec))
    same(kp, k, ke)
    assert (vp.double().cpu().numpy() == ve).all()
    assert device_status() == 0


def test_append_without_rotation_and_with_own_places():
    S, d, lens, T = 16, 64, [40, 33, 20], 20
    table = scattered(lens, S, 12, 5)
    q, k, v = tensors(3, T, 2, 2, d, "bf16", 6, False)
    args = (torch.as_tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    kp, vp = pools(12, 2, S, d, "bf16", 7)
    ke, ve = expected(k, v, kp, vp, table, lens, [T] * 3, S, lambda x: x.double().cpu().numpy())
    assert cache_append(k, v, kp, vp, *args) is None
    torch.cuda.synchronize()
    assert (kp.double().cpu().numpy() == ke).all() and (vp.double().cpu().numpy() == ve).all()
    plan = RopeAxes(d, (16, 16))
    place = (torch.tensor(lens)[:, None] - T + torch.arange(T)).int().expand(2, 3, T)
    ke, _ = expected(k, v, kp, vp, table, lens, [T] * 3, S, lambda x: rotated(x, place, (16, 16)))
    qo = cache_append(k, v, kp, vp, *args, rope=plan, q=q)
    torch.cuda.synchronize()
    same(kp, k, ke)
    same(qo, q, rotated(q, place, (16, 16)))


def test_append_of_bad_state_writes_nothing_there():
    S, d, T = 16, 64, 4
    lens, counts = [20, 3, 40, 500, 30], [4, 4, 5, 4, 4]  # 1: shorter than its count; 2: count > T; 3: past the table
    table = np.arange(5 * 3, dtype=np.int32).reshape(5, 3)
    table[4, 1] = 99  # the page its rows go to does not exist
    kp, vp = pools(15, 1, S, d, "bf16", 8)
    before = kp.clone()
    _, k, v = tensors(5, T, 1, 1, d, "bf16", 9, False)
    ints = dict(dtype=torch.int32, device="cuda")
    cache_append(k, v, kp, vp, torch.as_tensor(table).cuda(), torch.tensor(lens, **ints), counts=torch.tensor(counts, **ints))
    assert device_status() == -1 and device_status() == 0
    before[1, :, 0:4] = k[0]
    assert torch.equal(kp, before)


def test_a_given_stream_and_a_graph():
    plan = RopeAxes(128, (16, 24, 24))
    q, k, v = tensors(2, 5, 4, 2, 128, "bf16", 22, True)
    pos = draw_positions(3, 2, 5, 1000, 23)
    table, n = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4), torch.tensor([9, 30], dtype=torch.int32, device="cuda")
    want = rope(q, k, pos, plan)
    kp, vp = pools(8, 2, 8, 128, "bf16", 24)
    ke, ve = kp.clone(), vp.clone()
    qa = cache_append(k, v, ke, ve, table, n, rope=plan, positions=pos, q=q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = rope(q, k, pos, plan, stream=side)
    back = rope_backward(*got, pos, plan, stream=side)
    k2, v2 = kp.clone(), vp.clone()
    side.wait_stream(torch.cuda.current_stream())
    q2 = cache_append(k, v, k2, v2, table, n, rope=plan, positions=pos, q=q, stream=side)
    side.synchronize()
    for a, b in zip(got + (q2, k2, v2), want + (qa, ke, ve)):
        assert torch.equal(a, b)
    # turned back: a rounding to bf16 of each member of a pair each way
    assert ((back[0] - q).abs().float() <= 4 * 2.0 ** -8 * q.abs().max().float()).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g1 = rope(q, k, pos, plan)
        q3 = cache_append(k, v, kp, vp, table, n, rope=plan, positions=pos, q=q)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(g1 + (q3, kp, vp), want + (qa, ke, ve)):
        assert torch.equal(a, b)


def test_append_without_a_pool():
    _, k, v = tensors(2, 3, 2, 2, 64, "bf16", 20, False)
    e = torch.zeros(0, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    ints = dict(dtype=torch.int32, device="cuda")
    plan = RopeAxes(64, (32,))
    q, _, _ = tensors(2, 3, 2, 2, 64, "bf16", 21, False)
    qo = cache_append(k, v, e, e, torch.zeros(2, 1, **ints), torch.full((2,), 3, **ints), rope=plan, q=q)
    same(qo, q, rotated(q, torch.arange(3).expand(1, 2, 3), (32,)))
    assert device_status() == -1
    cache_append(k, v, e, e, torch.zeros(2, 1, **ints), torch.zeros(2, **ints), counts=torch.zeros(2, **ints))
    assert device_status() == 0


def test_refusals():
    plan = RopeAxes(64, (16, 16))
    q, k, v = tensors(2, 3, 2, 2, 64, "bf16", 13, False)
    pos = draw_positions(2, 2, 3, 10, 14)
    for bad in (lambda: rope(q, k.float(), pos, plan), lambda: rope(q.half(), None, pos, plan), lambda: rope(q, k, pos.long(), plan),
                lambda: rope(q, k, pos[:1], plan), lambda: rope(q[..., ::2], None, pos, RopeAxes(32, (16,))),
                lambda: rope(q, k, pos, RopeAxes(128, (16, 16))), lambda: rope(q, k, pos, None), lambda: rope(q[0], None, pos, plan),
                lambda: rope(q, k, pos, plan, q_out=q[:1].expand(2, 2, 3, 64)), lambda: rope(q.cpu(), None, pos, plan),
                lambda: cache_append(k, v, k, v, pos[0], pos[0, 0], q=q)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError):
        RopeAxes(64, (33,))
    with pytest.raises(ValueError):
        RopeAxes(64, ())
    with pytest.raises(CsaError):
        RopeAxes(64, (16,), base=-1.0)
    e, _ = rope(q[:0], None, pos[:, :0], plan)
    assert e.shape == (0, 2, 3, 64)


def test_an_output_without_its_input_is_refused():
    plan = RopeAxes(64, (16, 16))
    q, k, v = tensors(2, 3, 2, 2, 64, "bf16", 13, False)
    pos = draw_positions(2, 2, 3, 10, 14)
    pages = torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    lens = torch.full((2,), 3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        rope(q, None, pos, plan, k_out=torch.empty_like(k))
    for kw in ({}, {"rope": plan, "positions": pos}):
        with pytest.raises(ValueError):
            cache_append(k, v, pages, pages.clone(), table, lens, q_out=torch.empty_like(q), **kw)
