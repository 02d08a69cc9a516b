"""What the build does with and without torch, and after another torch: the compilers are stood in for."""

import os
import subprocess
import sys

import pytest

from blockwise_attn_ffn_bpt_b200 import build as b


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """The commands that the build runs, into an empty folder; each leaves its output there."""
    ran = []

    def run(cmd, **kw):
        ran.append(os.path.basename(cmd[0]))
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    for name in ("PKG", "LIB", "BINDING", "BUILT_FOR"):
        if hasattr(b, name):
            at = getattr(b, name)
            monkeypatch.setattr(b, name, str(tmp_path) if name == "PKG" else str(tmp_path / os.path.basename(at)))
    monkeypatch.setattr(b, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(b.subprocess, "run", run)
    return ran


def test_the_c_library_needs_no_torch(commands, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # as if it were not installed
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert commands == ["nvcc"] and b.up_to_date()
    assert "torch is not installed" in capsys.readouterr().err
    b.build()
    assert commands == ["nvcc"]


def test_another_torch_has_the_binding_built_again(commands, monkeypatch):
    b.build()
    assert commands == ["nvcc", "g++"] and b.up_to_date()
    b.build()
    assert commands == ["nvcc", "g++"]
    monkeypatch.setattr(b.importlib.metadata, "version", lambda name: "99.0")
    assert not b.up_to_date()
    b.build()
    assert commands == ["nvcc", "g++", "g++"] and b.up_to_date()
    b.build(force=True)
    assert commands == ["nvcc", "g++", "g++", "nvcc", "g++"]
