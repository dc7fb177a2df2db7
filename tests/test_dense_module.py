"""The binding's own module beside the library: what is built and what runs where it is not there."""
from __future__ import annotations

import os
import stat

import pytest
import torch

import tensor_core_loop_gb300 as tcl
from tensor_core_loop_gb300 import _build, dense
from test_dense_host import test_binding_refuses as refusals


@pytest.fixture(autouse=True)
def _fresh(monkeypatch):
    _build.build()
    monkeypatch.setattr(dense, "_native", None)


def absent(monkeypatch):
    monkeypatch.setattr(dense, "_native", False)


def test_module_is_built_and_used_here():
    if torch.version.cuda is None:
        pytest.skip("a PyTorch without GPUs")
    assert os.path.exists(_build.tensors_path()) and dense._load() is dense._native and dense._native


def without_compiler(monkeypatch, tmp_path):
    """g++ that fails as one without Python's headers does."""
    gxx = tmp_path / "g++"
    gxx.write_text("#!/bin/sh\necho 'fatal error: Python.h: No such file or directory' >&2\nexit 1\n")
    gxx.chmod(gxx.stat().st_mode | stat.S_IXUSR)
    which = _build.shutil.which
    monkeypatch.setattr(_build.shutil, "which", lambda name: str(gxx) if name == "g++" else which(name))
    monkeypatch.setattr(_build, "tensors_path", lambda: str(tmp_path / "_tensors.so"))


def test_library_is_built_where_the_module_cannot_be(monkeypatch, tmp_path):
    without_compiler(monkeypatch, tmp_path)
    monkeypatch.setattr(_build, "LIB_PATH", str(tmp_path / "lib.so"))   # (to be linked once more)
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert _build.build() == str(tmp_path / "lib.so")
    assert sorted(os.listdir(tmp_path)) == ["g++", "lib.so"]


def test_module_is_not_asked_of_a_pytorch_without_gpus(monkeypatch, tmp_path, recwarn):
    without_compiler(monkeypatch, tmp_path)
    monkeypatch.setattr(torch.version, "cuda", None)
    _build.build()
    assert not recwarn and os.listdir(tmp_path) == ["g++"]


def test_a_module_that_does_not_load_is_named_once(monkeypatch, tmp_path, recwarn):
    (tmp_path / "_tensors.so").write_bytes(b"not a library")
    monkeypatch.setattr(_build, "tensors_path", lambda: str(tmp_path / "_tensors.so"))
    for _ in range(3):
        with pytest.raises(ValueError, match="CUDA"):
            tcl.grad_norm([torch.zeros(4)])
    assert len([w for w in recwarn if str(tmp_path) in str(w.message)]) == 1


@pytest.mark.parametrize("where,name,value", [(torch, "__version__", "2.0.1"), (torch.version, "git_version", "0" * 40), (torch.version, "cuda", "12.9"),
                                              (torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)])
def test_a_module_of_another_pytorch_is_not_loaded(monkeypatch, where, name, value):
    """Exchanged for one with older file times or not."""
    there = _build.tensors_path()
    monkeypatch.setattr(where, name, value)
    assert _build.tensors_path() != there
    with pytest.warns(RuntimeWarning, match="without the binding's module"):
        assert dense._load() is False


def test_a_module_of_another_python_is_not_loaded(monkeypatch):
    there, var = _build.tensors_path(), _build.sysconfig.get_config_var
    monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda n: ".cpython-399.so" if n == "EXT_SUFFIX" else var(n))
    assert _build.tensors_path() != there
    with pytest.warns(RuntimeWarning, match="without the binding's module"):
        assert dense._load() is False


def test_binding_without_the_module_refuses(monkeypatch):
    absent(monkeypatch)
    refusals()
    for wrong, err in ((3, TypeError), (torch.zeros(4, 4).t()[1:], ValueError), (torch.eye(3).to_sparse(), ValueError)):
        with pytest.raises(err):
            tcl.grad_norm([torch.zeros(4), wrong])


@pytest.mark.gpu
def test_same_bits_without_the_module(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_gpu_dense import flat, operands, step
    ops = operands(61, 300, 136, 384, 2050)
    dense._load()
    few = [t[:5] for t in ops[:1]] + list(ops[1:5]) + [t[:5].contiguous() for t in ops[5:]]
    want = flat(step(*ops)) + flat(step(*few)) + [tcl.grad_norm(list(ops[:4])), *tcl.cross_entropy(ops[0], ops[4], ops[5])]
    absent(monkeypatch)
    got = flat(step(*ops)) + flat(step(*few)) + [tcl.grad_norm(list(ops[:4])), *tcl.cross_entropy(ops[0], ops[4], ops[5])]
    for a, b in zip(got, want, strict=True):
        assert torch.equal(a, b)
    assert tcl.last_device_error() == (0, 0)
