"""The build of the library and of the binding's compiled checks (no compiler is run
here): the checks are those of this interpreter and this torch, and the library does
not depend on them."""

import os
import subprocess
import sys
import types

import pytest
import torch

from paged_kv_attention_17_gb300 import _binding as B
from paged_kv_attention_17_gb300 import build as bld


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """An empty output folder, and a compiler that records its commands, creates
    their outputs, and fails for the sources named in ``bad``."""
    monkeypatch.setattr(bld, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(bld, "LIB", str(tmp_path / "libpkv.so"))
    if hasattr(bld, "CALLS"):
        monkeypatch.setattr(bld, "CALLS", str(tmp_path / "_calls.so"))
    t = types.SimpleNamespace(commands=[], bad="")

    def run(cmd, **kw):
        t.commands.append(cmd)
        if t.bad and any(str(x).endswith(t.bad) for x in cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="Python.h: no such file")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    return t


def built(t, name):
    return sum(any(str(x).endswith(name) for x in cmd) for cmd in t.commands)


def test_nothing_is_built_twice(tree):
    assert bld.build() == bld.LIB and os.path.exists(bld.LIB)
    assert built(tree, "calls.cpp") == 1 and built(tree, "decode.cu") == 1
    tree.commands.clear()
    bld.build()
    assert not tree.commands


@pytest.mark.parametrize("version", ["0.0.1", torch.__version__ + ".other"])
def test_another_torch_has_its_own_checks(tree, monkeypatch, version):
    bld.build()
    tree.commands.clear()
    monkeypatch.setattr(torch, "__version__", version)
    bld.build()
    assert built(tree, "calls.cpp") == 1
    assert built(tree, "decode.cu") == 0                  # the library does not know torch
    tree.commands.clear()
    monkeypatch.undo()


def test_another_interpreter_has_its_own_checks(tree, monkeypatch):
    bld.build()
    tree.commands.clear()
    config = bld.sysconfig.get_config_var
    monkeypatch.setattr(bld.sysconfig, "get_config_var",
                        lambda k: "cpython-399-other" if k in ("SOABI", "EXT_SUFFIX") else config(k))
    bld.build()
    assert built(tree, "calls.cpp") == 1 and built(tree, "decode.cu") == 0


def test_checks_of_another_torch_are_not_loaded(monkeypatch):
    monkeypatch.setattr(B, "_calls", None)
    assert B._load_calls() is not None                    # this torch's are there
    monkeypatch.setattr(B, "_calls", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(ImportError, match="not built"):
        B._load_calls()


def test_the_library_is_built_without_the_checks(tree):
    tree.bad = "calls.cpp"
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert bld.build() == bld.LIB
    assert os.path.exists(bld.LIB)
    tree.commands.clear()
    tree.bad = ""
    bld.build()                                           # tried again, and only that
    assert built(tree, "calls.cpp") == 1 and built(tree, "decode.cu") == 0


def test_the_library_is_built_without_torch(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert bld.build() == bld.LIB
    assert os.path.exists(bld.LIB) and built(tree, "decode.cu") == 1
    assert built(tree, "calls.cpp") == 0


def test_a_failing_library_is_an_error(tree):
    tree.bad = "decode.cu"
    with pytest.raises(RuntimeError, match="decode.cu"):
        bld.build()
    assert not os.path.exists(bld.LIB)
