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


def test_a_stale_binding_is_built_again(compilers, tmp_path, monkeypatch):
    """A changed header (the structs that binding and library share), binding
    source or recipe; a link that failed after the new library was in place;
    another torch."""
    commands, broken = compilers
    header = tmp_path / "include" / "ep_api.h"
    header.parent.mkdir()
    header.write_text("/* as it was */")
    monkeypatch.setattr(build, "ROOT", str(tmp_path))
    src = tmp_path / "moe_binding.cpp"
    src.write_text("// as it was")
    monkeypatch.setattr(build, "BINDING_SRC", str(src))
    build.build()
    assert build.binding_up_to_date()
    later = os.path.getmtime(build.BINDING) + 10
    for changed in (header, src):
        os.utime(changed, (later, later))
        broken.add("g++")                                    # the library gets there, the binding does not
        with pytest.raises(RuntimeError):
            build.build()
        broken.clear()
        assert not build.binding_up_to_date()
        os.utime(changed, (1, 1))
        assert build.binding_up_to_date()
    recipe = tmp_path / "build.py"
    recipe.write_text("")
    os.utime(recipe, (later, later))
    monkeypatch.setattr(build, "__file__", str(recipe))
    assert not build.binding_up_to_date()
    os.utime(recipe, (1, 1))
    import torch
    monkeypatch.setattr(torch, "__version__", "0.0")
    assert not build.binding_up_to_date()
    commands.clear()
    build.build_binding()
    assert commands and build.binding_up_to_date()
