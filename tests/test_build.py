"""The build's two products: the library, which needs nvcc alone, and the binding's
extension module, which fits one torch and may be missing."""
import os
import subprocess

import pytest
import torch

import memory_bound_glu_gb300 as mb
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


def test_the_library_without_the_module(tree):
    path, fails = tree
    build(path)
    fails.add("g++")
    with pytest.warns(UserWarning, match="not built"):
        build(path)
    assert (path / "lib.so").exists()
    assert not (path / "quick.so").exists() and not _build.quick_is_current()   # nor an old one


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
def test_the_binding_without_the_module(tree, monkeypatch, stale):
    """Every call goes to the library through binding.py, with its own errors."""
    path, _ = tree
    if stale:
        build(path)
        monkeypatch.setattr(torch, "__version__", "1.0")
    monkeypatch.setattr(binding, "_quick_module", None)
    with pytest.warns(UserWarning, match="another torch"):
        q = binding._quick()
    for name in ("glu_gemm", "wide_glu", "glu_gemm_backward", "add_rmsnorm_fp8", "glu_fp8", "matmul_fp8"):
        assert getattr(q, name)(1, 2, 3) is None
    assert binding._quick() is q
    with pytest.raises(TypeError, match="torch.Tensor"):
        mb.glu_gemm(None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        mb.matmul_fp8(torch.zeros(1, 128).to(mb.E4M3), None, None, None)


def test_the_built_module_says_what_it_is_for():
    assert _build.quick_is_current()
    assert binding._quick().__doc__ == _build.quick_stamp()
