"""build() with commands that are recorded instead of run: libcsa.so is built whatever becomes of the module
that calls it on torch tensors."""
import os
import subprocess

import pytest
import torch

from continuous_softmax_attention_gb300 import build as B


@pytest.fixture
def commands(monkeypatch, tmp_path):
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        broken = getattr(run, "broken", None)
        if broken and broken in " ".join(cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B, "ROOT", str(tmp_path))
    monkeypatch.setattr(B, "LIB_PATH", str(tmp_path / "libcsa.so"))
    monkeypatch.setattr(B, "TORCH_LIB_PATH", str(tmp_path / "_csa_torch.so"))
    return ran, run


def test_everything_is_built(commands, monkeypatch):
    monkeypatch.setattr(torch.version, "cuda", "13.0")
    ran, _ = commands
    assert B.build() == B.LIB_PATH
    assert os.path.exists(B.LIB_PATH) and os.path.exists(B.TORCH_LIB_PATH)
    assert len(ran) == len(B.SOURCES) + 3


def test_without_the_cuda_half_of_torch(commands, monkeypatch, capsys):
    monkeypatch.setattr(torch.version, "cuda", None)
    ran, _ = commands
    assert B.build() == B.LIB_PATH
    assert os.path.exists(B.LIB_PATH) and not os.path.exists(B.TORCH_LIB_PATH)
    assert len(ran) == len(B.SOURCES) + 1 and "left out" in capsys.readouterr().err


def test_a_module_that_does_not_compile(commands, monkeypatch):
    monkeypatch.setattr(torch.version, "cuda", "13.0")
    _, run = commands
    run.broken = B.TORCH_SOURCE
    with pytest.raises(RuntimeError, match=B.TORCH_SOURCE):
        B.build()
    assert os.path.exists(B.LIB_PATH)
