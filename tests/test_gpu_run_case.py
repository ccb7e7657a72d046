"""The runner for profilers does what its arguments ask for."""
import sys

import pytest

import continuous_softmax_attention_gb300 as csa
from continuous_softmax_attention_gb300 import run_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_paged_mode(mode, monkeypatch, capsys):
    seen, real = [], csa.decode_paged

    def spy(q, k, v, table, lens, k0=None, v0=None, *, mode=0, **kw):
        seen.append((mode, None if k0 is None else tuple(k0.shape), None if v0 is None else tuple(v0.shape)))
        return real(q, k, v, table, lens, k0, v0, mode=mode, **kw)

    monkeypatch.setattr(csa, "decode_paged", spy)
    monkeypatch.setattr(sys, "argv", ["run_case", "--paged", "--B", "2", "--H", "8", "--kv-heads", "2", "--T", "70", "--d", "64",
                                      "--page", "16", "--iters", "2", "--mode", str(mode)])
    run_case.main()
    assert [m for m, _, _ in seen] == [mode, mode]
    if mode == csa.GIVEN:
        assert all(k0 == v0 == (2, 64) for _, k0, v0 in seen)
    assert "ok status=0 short=0" in capsys.readouterr().out


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("draft", [0, 7])
def test_paged_kinds_and_drafts(kind, draft, monkeypatch, capsys):
    seen, real = [], csa.decode_tree
    monkeypatch.setattr(csa, "decode_tree", lambda q, k, *a, **kw: (seen.append((q.shape[2], k.dtype)), real(q, k, *a, **kw))[1])
    monkeypatch.setattr(sys, "argv", ["run_case", "--paged", "--B", "2", "--H", "8", "--kv-heads", "2", "--T", "70", "--d", "64",
                                      "--page", "16", "--iters", "3", "--kind", kind, "--draft", str(draft)])
    run_case.main()
    assert [n for n, _ in seen] == ([draft] * 3 if draft else [])
    assert "ok status=0 short=0" in capsys.readouterr().out
