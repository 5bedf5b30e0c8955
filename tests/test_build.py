"""The library builds and loads without the Python binding and what that needs;
stale files are not taken for current ones.  Compilers are stood in for."""
import os
import subprocess
import sys

import pytest

from combine_ep_layout_06_gb300 import _lib, build


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    """An empty build folder, and compilers that write what they are asked for;
    returns the commands and the set of programs that fail."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libep_gb300.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_moe.so"))
    commands, broken = [], set()

    def run(cmd, **kw):
        commands.append(cmd)
        if os.path.basename(cmd[0]) in broken:
            return subprocess.CompletedProcess(cmd, 1, "", "cannot")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build.subprocess, "run", run)
    return commands, broken


def test_the_library_builds_without_torch(compilers, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)          # as if it were not installed
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert {os.path.basename(c[0]) for c in compilers[0]} == {"nvcc"}


def test_the_library_is_in_place_when_the_binding_fails(compilers):
    commands, broken = compilers
    broken.add("g++")
    with pytest.raises(RuntimeError, match="moe_binding"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    broken.clear()
    commands.clear()
    build.build()                                            # only what is missing
    assert os.path.exists(build.BINDING)
    assert {os.path.basename(c[0]) for c in commands} == {"g++"}


def test_the_library_loads_without_the_binding(tmp_path, monkeypatch):
    _lib.load()
    monkeypatch.setattr(_lib, "_lib", None)
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_moe.so"))

    def never(*a, **kw):
        raise AssertionError("built again")
    for name in ("build", "build_library", "build_binding"):
        monkeypatch.setattr(build, name, never, raising=False)
    assert _lib.load().ep_status_str(0)
