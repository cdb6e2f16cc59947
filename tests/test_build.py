"""What build_library builds, with compilers that only record that they were called (no GPU, no toolkit)."""
import importlib
import os
import subprocess

import pytest

from exact_attention_18_gb300 import build as fab


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build module writing to an empty folder, through fake compilers; returns the targets made so far."""
    for name, path in (("BUILD_DIR", "_build"), ("LIB_DIR", "_lib")):
        monkeypatch.setattr(fab, name, str(tmp_path / path))
    monkeypatch.setattr(fab, "LIB_PATH", str(tmp_path / "_lib" / "libfa_gb300.so"))
    monkeypatch.setattr(fab, "BINDING_PATH", str(tmp_path / "_lib" / "_fa_binding.so"))
    monkeypatch.setattr(fab, "BINDING_FOR", str(tmp_path / "_build" / "fa_binding.for"))
    monkeypatch.setattr(fab, "nvcc", lambda: "/opt/nvcc/bin/nvcc")
    made = []

    def run(cmd, **kw):
        target = cmd[cmd.index("-o") + 1]
        made.append(os.path.basename(target).removesuffix(".tmp"))
        failed = made[-1] == "fa_binding.o" and getattr(run, "no_headers", False)
        if not failed:
            open(target, "w").close()
        return subprocess.CompletedProcess(cmd, int(failed), "", "no headers")

    monkeypatch.setattr(fab.subprocess, "run", run)
    return made, run


def test_library_and_binding_once(tree):
    made, _ = tree
    assert fab.build_library() == fab.LIB_PATH
    assert {"libfa_gb300.so", "_fa_binding.so", "fa_binding.o", "fa_api.o"} <= set(made)
    made.clear()
    fab.build_library()
    assert made == []
    fab.build_library(force=True)
    assert {"libfa_gb300.so", "_fa_binding.so"} <= set(made)


def test_library_alone_without_pytorch(tree, monkeypatch):
    made, _ = tree
    find = importlib.util.find_spec
    monkeypatch.setattr(fab.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert fab.build_library(verbose=True) == fab.LIB_PATH and os.path.exists(fab.LIB_PATH)
    assert "fa_binding.o" not in made and not os.path.exists(fab.BINDING_PATH)
    made.clear()
    fab.build_library()
    assert made == []


def test_library_is_there_when_the_binding_fails(tree):
    made, run = tree
    run.no_headers = True
    with pytest.raises(RuntimeError, match="no headers"):
        fab.build_library()
    assert os.path.exists(fab.LIB_PATH) and not os.path.exists(fab.BINDING_PATH)
    run.no_headers = False
    made.clear()
    fab.build_library()
    assert sorted(made) == ["_fa_binding.so", "fa_binding.o"]


def test_binding_of_another_pytorch_is_stale(tree, monkeypatch):
    made, _ = tree
    fab.build_library()
    made.clear()
    monkeypatch.setattr(fab.importlib.metadata, "version", lambda name: "0.0")
    fab.build_library()
    assert sorted(made) == ["_fa_binding.so", "fa_binding.o"]
