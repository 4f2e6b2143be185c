"""The build of the extension module: the library needs no torch, and a module that was built against another torch or
Python, whose tensors it would read by the wrong layout, is built anew and never used."""
import importlib.util
import os
import types

import pytest

import broadcast_implicit_gemm_gb300 as bg
from broadcast_implicit_gemm_gb300 import _build


@pytest.fixture
def apart(monkeypatch, tmp_path):
    """A build of one source elsewhere."""
    for name, at in (("BUILD", "_build"), ("LIB", "lib.so"), ("MODULE", "_layer.so"), ("STAMP", "_build/layer_for")):
        monkeypatch.setattr(_build, name, str(tmp_path / at))
    monkeypatch.setattr(_build, "sources", lambda: [os.path.join(_build.CSRC, "column_sums.cu")])
    return tmp_path


def torch_at(monkeypatch, root):
    find = importlib.util.find_spec
    found = root and types.SimpleNamespace(submodule_search_locations=[str(root)])
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: found if name == "torch" else find(name, *a))


@pytest.mark.parametrize("which", ["none", "without CUDA", "without headers"])
def test_the_library_needs_no_torch(monkeypatch, apart, which):
    root = None
    if which != "none":
        root = apart / "torch"
        (root / "lib").mkdir(parents=True)
        (root / "version.py").write_text("__version__ = '2.9.0'\ngit_version = 'abc'\ncuda = None\n")
        if which == "without headers":
            (root / "lib" / "libc10_cuda.so").touch()
    torch_at(monkeypatch, root)
    assert _build.build() == str(apart / "lib.so")
    assert os.path.exists(apart / "lib.so") and not os.path.exists(apart / "_layer.so")
    assert _build.up_to_date()


def test_a_module_of_another_torch_is_stale(monkeypatch, apart):
    _build.build()
    assert _build.up_to_date()
    built = os.path.getmtime(_build.LIB), os.path.getmtime(_build.MODULE)
    target = _build.layer_target()
    for other in (target.replace("torch ", "torch 1."), target.replace(" cpython", " xpython")):
        assert other != target
        monkeypatch.setattr(_build, "layer_target", lambda: other)
        assert not _build.up_to_date()
    monkeypatch.setattr(_build, "layer_target", lambda: target)
    assert _build.up_to_date()
    os.remove(_build.STAMP)
    assert not _build.up_to_date()
    _build.build()                   # the module alone
    assert _build.up_to_date() and os.path.getmtime(_build.LIB) == built[0] and os.path.getmtime(_build.MODULE) > built[1]


def test_a_library_that_is_there_does_not_wait_for_the_module(monkeypatch, apart):
    """A module that does not build is an error, after the library."""
    monkeypatch.setattr(_build, "_build_module", lambda: (_ for _ in ()).throw(RuntimeError("no module")))
    with pytest.raises(RuntimeError, match="no module"):
        _build.build()
    assert os.path.exists(apart / "lib.so")


def test_a_module_of_another_torch_is_refused(monkeypatch):
    torch = pytest.importorskip("torch")
    _build.build()
    monkeypatch.setattr(bg, "_layer_module", None)
    assert bg._layer().built_for == _build.layer_target()
    monkeypatch.setattr(bg, "_layer_module", None)
    monkeypatch.setattr(torch.version, "git_version", "another")
    with pytest.raises(RuntimeError, match="built for"):
        bg._layer()
    assert bg._layer_module is None
