"""When _ffn.so is compiled again."""
import os
import types

import pytest

torch = pytest.importorskip("torch")

from combine_route_count_gb300 import build as b  # noqa: E402


@pytest.fixture()
def compiles(tmp_path, monkeypatch):
    """build_ffn in a folder of its own, with a compiler that only writes its output; the commands it was given."""
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b, "LIB_FFN", str(tmp_path / "_ffn.so"))
    monkeypatch.setattr(b, "STAMP_FFN", str(tmp_path / "build" / "ffn.stamp"), raising=False)
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(b, "build", lambda: None)
    monkeypatch.setattr(b, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(b.subprocess, "run", run)
    return commands


def test_only_once(compiles):
    for _ in range(3):
        assert os.path.exists(b.build_ffn())
    assert len(compiles) == 1
    b.build_ffn(force=True)
    assert len(compiles) == 2


def test_again_for_another_torch(compiles, monkeypatch):
    b.build_ffn()
    monkeypatch.setattr(torch, "__version__", "0.0.test")
    b.build_ffn()
    assert len(compiles) == 2
    b.build_ffn()
    assert len(compiles) == 2


def test_again_without_its_record(compiles):
    b.build_ffn()
    os.remove(b.STAMP_FFN)
    b.build_ffn()
    assert len(compiles) == 2
