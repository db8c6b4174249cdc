"""What is built when the Python binding's module cannot be, and when it is out of date."""

from __future__ import annotations

import pytest
import torch

from selective_state_update_02_gb300 import _build
import selective_state_update_02_gb300 as ssu


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """A build of one small unit into a folder of its own."""
    monkeypatch.setattr(_build, "OBJDIR", tmp_path / "objects")
    monkeypatch.setattr(_build, "LIB", tmp_path / "libssu.so")
    monkeypatch.setattr(_build, "MARSHAL", tmp_path / "_marshal.so")
    monkeypatch.setattr(_build, "SOURCES", [_build.CSRC / "ssu_host.cpp"])
    return tmp_path


def fails(out):
    return ["false"]


def is_missing(out):
    return ["/nowhere/g++"]


def has_no_torch(out):
    raise ImportError("torch")


@pytest.mark.parametrize("compiler", [fails, is_missing, has_no_torch])
def test_the_library_does_not_need_the_binding(elsewhere, monkeypatch, compiler):
    monkeypatch.setattr(_build, "marshal_command", compiler)
    (elsewhere / "_marshal.so").write_bytes(b"of other sources")
    with pytest.warns(UserWarning, match="_marshal.so could not be built"):
        assert _build.build(force=True) == elsewhere / "libssu.so"
    assert (elsewhere / "libssu.so").exists()
    assert not (elsewhere / "_marshal.so").exists() and _build.stale()
    # the next build tries the binding again and leaves the library as it is
    before = (elsewhere / "libssu.so").stat().st_mtime_ns
    monkeypatch.setattr(_build, "marshal_command", lambda out: ["touch", str(out)])
    _build.build()
    assert (elsewhere / "libssu.so").stat().st_mtime_ns == before and not _build.stale()


def test_a_call_that_needs_the_binding_says_so(monkeypatch, tmp_path):
    monkeypatch.setattr(ssu, "_bound", None)
    monkeypatch.setattr(ssu, "MARSHAL_PATH", tmp_path / "_marshal.so")
    with pytest.raises(RuntimeError, match="_marshal.so is missing"):
        ssu.ssu_attend(0, None, None, None, None, None, None, stream=0)


def test_a_library_that_does_not_compile_is_an_error(elsewhere, monkeypatch):
    monkeypatch.setattr(_build, "compile_command", lambda src, obj, extra=None: ["false"])
    monkeypatch.setattr(_build, "marshal_command", lambda out: ["touch", str(out)])
    with pytest.raises(Exception, match="nvcc"):
        _build.build(force=True)
    assert not (elsewhere / "libssu.so").exists()


def test_the_binding_is_built_again_for_another_torch(elsewhere, monkeypatch):
    monkeypatch.setattr(_build, "marshal_command", lambda out: ["touch", str(out)])
    _build.build()
    assert not _build.stale()
    monkeypatch.setattr(torch, "__version__", "0.1")
    assert _build.stale()
    monkeypatch.setattr(ssu, "_bound", None)
    monkeypatch.setattr(ssu, "MARSHAL_PATH", elsewhere / "_marshal.so")
    with pytest.raises(RuntimeError, match="was built for torch .* build it again"):
        ssu.ssu_attend(0, None, None, None, None, None, None, stream=0)
    before = (elsewhere / "libssu.so").stat().st_mtime_ns
    _build.build()
    assert not _build.stale() and (elsewhere / "libssu.so").stat().st_mtime_ns == before
