"""The build of the library does not hang on the extension module beside it."""
from __future__ import annotations

import os

import pytest

pytest.importorskip("torch")

from reduce_copy_rank_gb300 import _build  # noqa: E402


@pytest.fixture(params=["/bin/false", "/nonexistent/compiler"])
def no_binding(request, monkeypatch, tmp_path):
    """The module's place is empty and its compiler fails or is not there."""
    _build.build()
    monkeypatch.setenv("CXX", request.param)
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_binding.so"))
    return tmp_path


def test_an_up_to_date_library_is_returned(no_binding):
    with pytest.warns(RuntimeWarning, match="extension module"):
        assert _build.build() == _build.LIB


def test_the_library_is_linked(no_binding, monkeypatch):
    monkeypatch.setattr(_build, "LIB", str(no_binding / "lib.so"))
    monkeypatch.setattr(_build, "OBJDIR", str(no_binding / "objects"))
    one = os.path.join(_build.CSRC, "dc_delay.cu")  # (a unit that compiles quickly)
    monkeypatch.setattr(_build, "sources", lambda: [one])
    with pytest.warns(RuntimeWarning, match="extension module"):
        assert _build.build() == _build.LIB
    assert os.path.getsize(_build.LIB) > 0


def test_a_module_of_older_sources_does_not_stay(no_binding):
    old = no_binding / "_binding.so"
    old.write_bytes(b"old")
    os.utime(old, (1, 1))
    with pytest.warns(RuntimeWarning):
        _build.build()
    assert not old.exists()


def test_an_up_to_date_library_needs_no_cuda_compiler(no_binding, monkeypatch):
    def none():
        raise RuntimeError("nvcc not found")

    monkeypatch.setattr(_build, "_nvcc", none)
    with pytest.warns(RuntimeWarning, match="nvcc not found"):
        assert _build.build() == _build.LIB


def test_the_module_alone_raises(no_binding):
    with pytest.raises((RuntimeError, OSError)):
        _build.build_binding()
