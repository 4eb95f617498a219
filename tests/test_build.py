"""The library and the binding's compiled module apart: the library is built and loaded without the module, and a module
built for another torch or Python is neither taken for current nor used."""

import os
import subprocess
import sys
import types

import pytest

from _util import ensure_built
from exact_attention_06_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_the_library_loads_without_the_compiled_module():
    ensure_built()
    _python("""
import ctypes, sys
sys.modules["exact_attention_06_gb300._calls"] = None  # an import of it fails
from exact_attention_06_gb300 import fattn
L = fattn.lib()
assert L.fa_fwd(None, None, None, None, None, 1, 1, 1, 64, 0.1, 0, None) == fattn.FA_ERR_INVALID_ARG
assert fattn.fa_rope_axes_plan(64, (32,)).d == 64
for call in (lambda: fattn.fa_cross_fwd(None, None, None, None, None, 0.1),
             lambda: fattn.fa_cross_bwd(None, None, None, None, None, None, None, None, None, 0.1),
             lambda: fattn.fa_rope_axes(None, None, None, None),
             lambda: fattn.fa_rope_axes_paged(None, None, None, None, None, None, None, None, None, None)):
    try:
        call()
    except fattn.FattnError as e:
        assert e.status == fattn.FA_ERR_CUDA and "_calls.so" in str(e) and "build" in str(e), e
    else:
        raise AssertionError("not refused")
""")


@pytest.mark.parametrize("built_for", ["torch 1.0, .cpython-312-x86_64-linux-gnu.so", None])
def test_a_module_built_for_something_else_is_not_used(built_for):
    ensure_built()
    _python(f"""
import sys, types
m = types.ModuleType("exact_attention_06_gb300._calls")
m.bind = None  # (not reached)
if {built_for!r}: m.BUILT_FOR = {built_for!r}
import exact_attention_06_gb300 as package
sys.modules[m.__name__] = package._calls = m
from exact_attention_06_gb300 import fattn
fattn.lib()
try:
    fattn.fa_rope_axes(None, None, None, None)
except fattn.FattnError as e:
    assert "was built for" in str(e), e
else:
    raise AssertionError("not refused")
""")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build's outputs in a directory of their own, and its compilers as a list of the commands they were given."""
    for name, file in (("LIB", "libfattn.so"), ("CALLS", "_calls.so"), ("BUILD", "_build"),
                       ("CALLS_STAMP", "_build/_calls.stamp")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    t = types.SimpleNamespace(commands=[], fails=lambda cmd: False)

    def run(cmd, **kw):
        t.commands.append(cmd)
        if t.fails(cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setenv("CXX", "g++")
    return t


def test_what_is_current_is_not_built_again(tree):
    assert not build.up_to_date()
    assert build.build() == build.LIB
    assert len(tree.commands) == len(build.SOURCES) + 2 and build.up_to_date()
    build.build()
    assert len(tree.commands) == len(build.SOURCES) + 2


@pytest.mark.parametrize("what", ["torch", "place", "python", "compiler"])
def test_another_torch_or_python_makes_the_module_stale(tree, monkeypatch, what):
    import torch
    build.build()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "9.9.9")
    elif what == "place":
        monkeypatch.setattr(torch, "__file__", "/elsewhere/torch/__init__.py")
    elif what == "python":
        monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: ".cpython-399.so")
    else:
        monkeypatch.setenv("CXX", "c++")
    assert not build.up_to_date()
    before = len(tree.commands)
    build.build()
    assert len(tree.commands) == before + 1  # the module alone
    assert build.up_to_date()


def test_the_library_is_linked_when_the_module_does_not_compile(tree):
    tree.fails = lambda cmd: build.CALLS_SRC in cmd
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS) and not build.up_to_date()
    tree.fails = lambda cmd: False
    before = len(tree.commands)
    build.build()
    assert len(tree.commands) == before + 1 and build.up_to_date()


def test_the_library_is_linked_without_a_host_compiler(tree, monkeypatch):
    run = build.subprocess.run

    def no_host_compiler(cmd, **kw):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        return run(cmd, **kw)

    monkeypatch.setattr(build.subprocess, "run", no_host_compiler)
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        build.build()
    assert os.path.exists(build.LIB)
