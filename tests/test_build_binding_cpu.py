"""The native Python entries are rebuilt for another torch, and one built for another is not loaded."""
import os

import pytest
import torch

from block_sparse_attention_oam_b200 import build as B
from block_sparse_attention_oam_b200 import stem as S


@pytest.fixture
def other_torch(tmp_path, monkeypatch):
    """The module as it was built here, seen from another torch version."""
    B.build_binding()
    path = tmp_path / "stem_binding.so"
    path.write_bytes(open(B.BINDING, "rb").read())
    os.utime(path)
    monkeypatch.setattr(B, "BINDING", str(path))
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    return path


def test_the_module_here_fits():
    B.build_binding()
    assert B.binding_fits()
    assert len(S._binding()) == 4


def test_another_torch_is_not_given_this_module(other_torch, monkeypatch):
    monkeypatch.setattr(S, "_native", None)
    with pytest.raises(RuntimeError, match="another torch"):
        S._binding()
    assert S._native is None


def test_another_torch_rebuilds(other_torch, monkeypatch):
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").write(B.binding_tag().encode() + b"\0")
        return type("R", (), dict(returncode=0, stdout="", stderr=""))

    monkeypatch.setattr(B.subprocess, "run", run)
    B.build_binding()
    assert len(ran) == 1 and any("9.9.9" in a for a in ran[0])
    B.build_binding()
    assert len(ran) == 1                     # and then it is up to date
