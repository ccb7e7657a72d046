"""The status words of the paged cache's and rotary kernels, one per translation unit, are read and cleared together
(csa_device_status)."""
import threading

import pytest
import torch

from continuous_softmax_attention_gb300 import (cache_accept, cache_append, cache_free, cache_read, decode_paged, decode_tree,
                                                device_status)
from draft_util import KINDS

pytestmark = pytest.mark.gpu
INT = dict(dtype=torch.int32, device="cuda")


def wrong_calls():
    """A call with a length or page out of range for every unit that has a word."""
    d, S, bf = 64, 16, torch.bfloat16
    table, lens = torch.tensor([[0, 7]], **INT), torch.tensor([20], **INT)  # the second page does not exist
    calls = {}
    for kind in ("bf16", "e4m3", "int8"):
        pool = torch.zeros(2, 1, S, d, device="cuda").to(KINDS.get(kind, bf))
        kw = {} if kind == "bf16" else dict(row_scales=torch.ones(2, 1, S, 2, device="cuda"))
        new = torch.zeros(1, 1, 1, d, dtype=bf, device="cuda")
        calls[f"append {kind}"] = lambda pool=pool, kw=kw, new=new: cache_append(new, new, pool, pool, table, lens, **kw)
        calls[f"read {kind}"] = lambda pool=pool, kw=kw: cache_read(pool, pool, table, lens, 20, **kw)
        calls[f"step {kind}"] = lambda pool=pool, kw=kw: decode_paged(new[:, 0], pool, pool, table, lens, **kw)
        for heads in (1, 20):  # a draft of one token on page 0 of a sequence whose earlier rows are lost, and the reverse
            q = torch.zeros(1, heads, 1, d, dtype=bf, device="cuda")
            calls[f"tree {kind} {heads}"] = lambda q=q, pool=pool, kw=kw: decode_tree(q, pool, pool, table, lens, **kw)
            calls[f"past {kind} {heads}"] = lambda q=q, pool=pool, kw=kw: decode_tree(q, pool, pool, table.flip(1), lens, **kw)
    books = [torch.ones(2, **INT), table.clone(), lens.clone()]
    calls["free"] = lambda: cache_free(*[t.clone() for t in books], S, torch.tensor([5], **INT))
    calls["accept"] = lambda: cache_accept(*[t.clone() for t in books], S, torch.tensor([9], **INT), 3)
    return calls


def test_every_word_is_reported_once():
    device_status()
    for name, call in wrong_calls().items():
        call()
        assert device_status() == -1, name
        assert device_status() == 0, name


def test_words_together_are_one_report():
    device_status()
    for call in wrong_calls().values():
        call()
    assert device_status() == -1 and device_status() == 0


def test_two_threads_lose_no_report():
    """Of two readers at once one gets the report."""
    device_status()
    call = wrong_calls()["read e4m3"]
    for _ in range(50):
        call()
        torch.cuda.synchronize()
        got = []
        readers = [threading.Thread(target=lambda: got.append(device_status())) for _ in range(2)]
        for t in readers:
            t.start()
        for t in readers:
            t.join()
        assert sorted(got) == [-1, 0]
