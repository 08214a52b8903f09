"""The build's two products: the library, and the binding's extension module, which
fits one torch."""
import os
import subprocess

import pytest
import torch

from memory_bound_glu_gb300 import _build, binding


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build whose compilers are fakes that write their output; fails: names of those that fail."""
    fails = set()

    def run(cmd, check=False, **kw):
        name = os.path.basename(cmd[0])
        if name in fails:
            raise subprocess.CalledProcessError(1, cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(next((a for a in cmd if a.startswith("-DMBGLU_BUILT_FOR=")), "").strip('"').partition('"')[2] + "\0")

    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(_build.subprocess, "run", run)
    for name, file in (("LIB", "lib.so"), ("QUICK", "quick.so")):
        monkeypatch.setattr(_build, name, str(tmp_path / file))
    return tmp_path, fails


def build(tmp_path):
    return _build.build(str(tmp_path / "lib.so"))


def test_both_products(tree):
    path, _ = tree
    assert _build.needs_build(str(path / "lib.so"))
    build(path)
    assert (path / "lib.so").exists() and (path / "quick.so").exists()
    assert _build.quick_is_current() and not _build.needs_build(str(path / "lib.so"))


def test_a_library_that_fails_is_an_error(tree):
    path, fails = tree
    fails.add("nvcc")
    with pytest.raises(subprocess.CalledProcessError):
        build(path)


def test_a_module_of_another_torch_is_stale(tree, monkeypatch):
    path, _ = tree
    build(path)
    monkeypatch.setattr(torch, "__version__", "1.0")
    assert not _build.quick_is_current() and _build.needs_build(str(path / "lib.so"))


@pytest.mark.parametrize("stale", [False, True])
def test_the_binding_loads_no_such_module(tree, monkeypatch, stale):
    path, _ = tree
    if stale:
        build(path)
        monkeypatch.setattr(torch, "__version__", "1.0")
    monkeypatch.setattr(binding, "_quick_module", None)
    with pytest.raises(RuntimeError, match="another torch"):
        binding._quick()


def test_the_built_module_says_what_it_is_for():
    assert _build.quick_is_current()
    assert binding._quick().__doc__ == _build.quick_stamp()
