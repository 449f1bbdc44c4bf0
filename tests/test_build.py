"""The build's order and its idea of what is up to date, with the compilers
replaced by a stand-in (nothing is compiled)."""
import os
import types
import warnings

import pytest

from ring_all_reduce_rar_gb300 import _build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """An empty build folder, and compilers that only write their output file;
    `fail` names a word of the commands that end with an error."""
    log = types.SimpleNamespace(commands=[], fail=None)

    def run(cmd, **kw):
        log.commands.append(cmd)
        if log.fail and any(log.fail in word for word in cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="refused")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("x")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(_build, "subprocess", types.SimpleNamespace(run=run))
    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(_build, "LIB_PATH", str(tmp_path / "librar.so"))
    monkeypatch.setattr(_build, "TORCH_OPS_PATH", str(tmp_path / "_torch_ops.so"))
    return log


binding = pytest.mark.skipif(_build.binding_lacks() is not None, reason="the binding cannot be built here")


@binding
@pytest.mark.parametrize("fail", ["torch_ops.cpp", "-ltorch_python"])
def test_a_binding_that_fails_leaves_the_library(tree, fail):
    """The C library needs nothing of the binding: it is there when the binding's
    compilation or link fails, which is still reported."""
    tree.fail = fail
    with pytest.raises(RuntimeError, match="torch_ops"):
        _build.build()
    assert os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.TORCH_OPS_PATH)


@pytest.mark.parametrize("what", ["g++", "Python.h", "libc10_cuda.so"])
def test_without_the_bindings_needs_the_library_is_built(tree, monkeypatch, what):
    """A machine that lacks what only the binding needs builds the library."""
    which, exists = _build.shutil.which, os.path.exists
    monkeypatch.setattr(_build.shutil, "which", lambda name: None if name == what else which(name))
    monkeypatch.setattr(_build.os.path, "exists", lambda path: os.path.basename(path) != what and exists(path))
    with pytest.warns(UserWarning, match="_torch_ops.so is not built"):
        _build.build()
    assert exists(_build.LIB_PATH) and not exists(_build.TORCH_OPS_PATH)
    assert not any("torch_ops.cpp" in word for cmd in tree.commands for word in cmd)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert _build.up_to_date()


@binding
def test_both_are_built(tree):
    _build.build()
    assert os.path.exists(_build.LIB_PATH) and os.path.exists(_build.TORCH_OPS_PATH) and _build.up_to_date()
    n = len(tree.commands)
    _build.build()
    assert len(tree.commands) == n


@binding
def test_another_torch_is_seen(tree, monkeypatch):
    """The binding belongs to the torch that it was built against."""
    _build.build()
    assert _build.up_to_date()
    monkeypatch.setattr(_build, "_torch_version", lambda: "another version")
    assert not _build.up_to_date()
    _build.build()
    assert _build.up_to_date()


def test_torch_version_without_importing_it():
    torch = pytest.importorskip("torch")
    assert torch.__version__ in _build._torch_version()
