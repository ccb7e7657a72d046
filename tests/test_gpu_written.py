"""What the paged cache's and the rotary positions' calls write raises its version, so that autograd refuses
to go backward through a saved tensor that was overwritten; what they only read does not."""
import pytest
import torch

import continuous_softmax_attention_gb300 as csa

pytestmark = pytest.mark.gpu


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def versions(call, written, read):
    tensors = list(written) + list(read)
    before = [t._version for t in tensors]
    call()
    after = [t._version for t in tensors]
    for i, (a, b) in enumerate(zip(before, after)):
        assert b > a if i < len(written) else b == a, i


def test_versions_of_written_tensors():
    plan = csa.RopeAxes(64, (16, 16))
    bf = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)
    q, k, v, pos = bf(2, 4, 3, 64), bf(2, 2, 3, 64), bf(2, 2, 3, 64), torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    kp, vp = bf(8, 2, 8, 64), bf(8, 2, 8, 64)
    refs, table, lens, counts = torch.zeros(8, dtype=torch.int32, device="cuda"), torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), ints(0, 0), ints(3, 0)
    short, rows = ints(7), ints(1, -1)
    versions(lambda: csa.rope(q, k, pos, plan, q_out=qo, k_out=ko), [qo, ko], [q, k, pos])
    versions(lambda: csa.rope_backward(q, None, pos, plan, q_out=q), [q], [pos])
    versions(lambda: csa.cache_reserve(refs, table, lens, 8, counts, shortfall=short), [refs, table, lens, short], [counts])
    versions(lambda: csa.cache_append(k, v, kp, vp, table, lens, counts=counts, rope=plan, positions=pos, q=q, q_out=qo),
             [kp, vp, qo], [k, v, q, table, lens, counts, pos])
    versions(lambda: csa.cache_fork(refs, table, lens, 8, ints(0), rows[:1]), [refs, table, lens], [rows])
    versions(lambda: csa.cache_copy_pages(kp, vp, ints(0), ints(3)), [kp, vp], [])
    versions(lambda: csa.cache_copy_pages(kp, None, ints(0), ints(3)), [kp], [vp])
    out, lse = torch.empty_like(q[:, :, 0]).contiguous(), torch.empty(2, 4, device="cuda")
    ws = torch.empty(csa.decode_paged_workspace_bytes(2, 4, 2, 64), dtype=torch.uint8, device="cuda")
    q1 = q[:, :, 0].contiguous()
    versions(lambda: csa.decode_paged(q1, kp, vp, table, lens, out=out, lse=lse, workspace=ws), [out, lse, ws], [q1, kp, vp, table, lens])
    versions(lambda: csa.cache_free(refs, table, lens, 8, rows), [refs, table, lens], [rows])
    versions(lambda: csa.cache_compact(refs, table, lens, 8), [refs, table], [lens])
    assert csa.device_status() == 0


def test_a_saved_tensor_rotated_in_place_is_refused():
    plan = csa.RopeAxes(64, (32,))
    a = torch.randn(1, 2, 5, 64, device="cuda", requires_grad=True)
    b = a * 1.0
    loss = (b * b).sum()  # saves b
    csa.rope(b.detach(), None, torch.arange(5, dtype=torch.int32, device="cuda"), plan, q_out=b.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_tensors_made_in_inference_mode_are_taken():
    plan = csa.RopeAxes(64, (32,))
    with torch.inference_mode():
        x = torch.randn(1, 2, 5, 64, device="cuda")
        want = csa.rope(x, None, torch.arange(5, dtype=torch.int32, device="cuda"), plan)[0]
    csa.rope(x, None, torch.arange(5, dtype=torch.int32, device="cuda"), plan, q_out=x)
    assert torch.equal(x, want)
