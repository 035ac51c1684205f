"""What the build compiles and when: the commands it would run, on made-up object files.  No compiler, no GPU."""
import os
import runpy
import sys
import types

import pytest

from sparse_attention_lightning_score_b200 import build as b


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """Runs of a command are recorded, and write the file that it would."""
    seen = []

    def run(cmd, **kw):
        seen.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "nvcc", lambda: "nvcc")
    for name, at in [("BUILD_DIR", "_build"), ("LIB", "libli.so"), ("BIND", "_bind.so"), ("BIND_STAMP", "_build/bind.txt")]:
        monkeypatch.setattr(b, name, str(tmp_path / at))
    return seen


def _by(commands, tool):
    return [c for c in commands if os.path.basename(c[0]) == tool]


def test_the_library_alone_needs_no_torch(monkeypatch, commands):
    monkeypatch.setitem(sys.modules, "torch", None)          # (an import of it raises)
    b.build(bind=False)
    assert len(_by(commands, "nvcc")) == len(commands) == len(b._sources()) + 1 and os.path.exists(b.LIB)


def test_the_build_file_runs_without_the_package(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.delitem(sys.modules, "sparse_attention_lightning_score_b200")
    alone = runpy.run_path(b.__file__, run_name="alone")
    assert alone["LIB"] == b.LIB and "sparse_attention_lightning_score_b200" not in sys.modules


def test_without_torch_the_library_is_built_before_the_binding_is_refused(monkeypatch, commands):
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.raises(RuntimeError, match="abi-only"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BIND)


def test_a_binding_that_does_not_compile_leaves_the_library(monkeypatch, commands):
    run = b.subprocess.run
    monkeypatch.setattr(b.subprocess, "run", lambda cmd, **kw: types.SimpleNamespace(
        returncode=1, stdout="", stderr="no Python.h") if cmd[0] == "g++" else run(cmd, **kw))
    with pytest.raises(RuntimeError, match="no Python.h"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BIND)


def test_the_binding_follows_torch(monkeypatch, commands):
    import torch
    b.build()
    assert len(_by(commands, "g++")) == 2 and os.path.exists(b.BIND)
    commands.clear()
    b.build()
    assert commands == []
    monkeypatch.setattr(torch, "__version__", "999.0")       # another torch, no date of ours has changed
    b.build()
    assert len(_by(commands, "g++")) == len(commands) == 2
    commands.clear()
    b.build()
    assert commands == []


def test_a_binding_whose_link_failed_is_made_again(monkeypatch, commands):
    run = b.subprocess.run
    with monkeypatch.context() as m:
        m.setattr(b.subprocess, "run", lambda cmd, **kw: types.SimpleNamespace(
            returncode=1, stdout="", stderr="link") if cmd[0] == "g++" and "-shared" in cmd else run(cmd, **kw))
        with pytest.raises(RuntimeError, match="link"):
            b.build()
    assert not os.path.exists(b.BIND_STAMP)
    b.build()
    assert os.path.exists(b.BIND) and os.path.exists(b.BIND_STAMP)
