"""The build where the Python binding's requirements are not met: libaf.so alone, as C callers need it."""
import os

import pytest

from video_generation_b200 import build as B


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The built library, and a binding path of its own."""
    B.build()
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_binding.so"))
    return str(tmp_path / "_binding.so")


def _without_torch(monkeypatch):
    find = B.importlib.util.find_spec
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def _without_compiler(monkeypatch):
    which = B.shutil.which
    monkeypatch.setattr(B.shutil, "which", lambda name, *a: None if name == "g++" else which(name, *a))


def _without_headers(monkeypatch):
    monkeypatch.setattr(B.sysconfig, "get_paths", lambda *a: {"include": "/nowhere"})


@pytest.mark.parametrize("lacking,what", [(_without_torch, "PyTorch"), (_without_compiler, "g++"),
                                          (_without_headers, "headers")])
def test_the_library_is_built_without_the_binding(elsewhere, monkeypatch, capsys, lacking, what):
    lacking(monkeypatch)
    assert B.build() == B.LIB and os.path.exists(B.LIB)
    assert not os.path.exists(elsewhere) and what in capsys.readouterr().err
    with open(elsewhere, "wb"):                             # a binding of older sources does not stay
        os.utime(elsewhere, (1, 1))
    B.build()
    assert not os.path.exists(elsewhere)


def test_the_binding_is_built_where_it_can_be(elsewhere):
    assert B._binding_lacks(B._torch_dir()) is None
    B._build_binding(os.path.dirname(os.path.dirname(os.path.realpath(B.nvcc()))), False, False)
    assert os.path.getsize(elsewhere) > 0
