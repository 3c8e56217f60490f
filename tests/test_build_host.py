"""The build's order, with the compilers' runs replaced by a fake: the C library
needs nvcc alone."""
import importlib.util
import os
import subprocess

import pytest

from vocabulary_cross_entropy_pass_gb300 import build


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """A build into an empty folder whose compilers touch their outputs; `fails` names one that does not."""
    (tmp_path / "bin").mkdir()
    cc = tmp_path / "bin" / "nvcc"
    cc.write_text("")
    monkeypatch.setattr(build, "nvcc", lambda: str(cc))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libgbce.so"))
    monkeypatch.setattr(build, "EXT", str(tmp_path / "_gbce_torch.so"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    state = {"fails": None, "ran": []}

    def run(cmd, **kw):
        state["ran"].append(cmd)
        ok = state["fails"] is None or state["fails"] not in " ".join(cmd)
        if ok:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0 if ok else 1, "", "refused")

    monkeypatch.setattr(build.subprocess, "run", run)
    return state


def test_both_are_built(tools):
    assert not build.up_to_date()
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.EXT)
    assert build.up_to_date()
    n = len(tools["ran"])
    build.build()
    assert len(tools["ran"]) == n


def test_the_library_is_linked_where_the_host_module_fails(tools):
    tools["fails"] = "ce_torch.cpp"
    with pytest.raises(RuntimeError, match="ce_torch.cpp"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.EXT)
    assert not build.up_to_date()


def test_the_library_is_built_without_torch(tools, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.EXT)
    assert build.up_to_date()
    assert not any("g++" in cmd[0] for cmd in tools["ran"])


def test_a_kernel_that_fails_leaves_no_library(tools):
    tools["fails"] = "ce_norm.cu"
    with pytest.raises(RuntimeError, match="ce_norm.cu"):
        build.build()
    assert not os.path.exists(build.LIB)
