"""The build's own logic, with a stand-in for the compilers: what is built where something is missing, and
what counts as up to date."""

import os
import sys
import types

import pytest
import torch

from lm_head_linear_gb300 import build as b
from lm_head_linear_gb300 import ops


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build folder of its own, compilers that write their -o, and the commands they got."""
    t = types.SimpleNamespace(ran=[], fails=lambda cmd: False)

    def run(cmd, verbose):
        t.ran.append(cmd)
        if t.fails(cmd):
            raise RuntimeError("the compiler's text")
        with open(cmd[cmd.index("-o") + 1], "w") as fh:
            fh.write("built")

    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "nvcc_path", lambda: "/cuda/bin/nvcc")
    monkeypatch.setattr(b, "LIB_DIR", str(tmp_path))
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / "libflce.so"))
    monkeypatch.setattr(b, "OPS_PATH", str(tmp_path / "flce_ops.so"))
    t.built = lambda: (os.path.exists(b.LIB_PATH), os.path.exists(b.OPS_PATH))
    return t


def test_both_are_built_once(tree):
    assert b.build() == b.LIB_PATH and tree.built() == (True, True)
    assert len(tree.ran) == len(b.SOURCES) + 3  # and two links and the module's source
    b.build()
    assert len(tree.ran) == len(b.SOURCES) + 3


@pytest.mark.parametrize("missing", ["torch's build helpers", "headers", "libraries"])
def test_the_library_builds_without_the_module(tree, monkeypatch, missing):
    """As it did when there was only the library; an older module does not stay behind."""
    b.build()
    if missing == "torch's build helpers":
        def commands(obj, out):
            raise ImportError("no cpp_extension")
        monkeypatch.setattr(b, "ops_commands", commands)
    else:
        last = b.OPS_SOURCE if missing == "headers" else "-ltorch_python"
        tree.fails = lambda cmd: last in cmd
    os.remove(b.LIB_PATH)
    with pytest.warns(UserWarning, match="could not be"):
        assert b.build() == b.LIB_PATH
    assert tree.built() == (True, False)


def test_a_library_that_fails_to_build_raises(tree):
    tree.fails = lambda cmd: b.SOURCES[1] in cmd
    with pytest.raises(RuntimeError, match="compiler's text"):
        b.build()
    assert tree.built() == (False, False)


def test_a_module_built_for_another_torch_is_stale(tree, monkeypatch):
    """torch's C++ interface has no stable ABI: a module built against another version is built again, and not loaded."""
    b.build()
    assert b.up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not b.up_to_date()
    monkeypatch.setattr(ops, "_OPS", None)
    monkeypatch.setattr(ops, "OPS_PATH", b.OPS_PATH)
    monkeypatch.setattr(ops, "load_library", lambda: None)
    with pytest.raises(RuntimeError, match="build it again"):
        ops.load_operators()
    b.build()
    assert b.up_to_date()
    os.remove(b.OPS_PATH + ".for")
    assert not b.up_to_date()
