"""CPU: the libraries are built where the binding's compiled short way cannot be."""
import subprocess

import pytest

from fp8_fine_grained_fp8bs_amd import build


@pytest.fixture
def traced(monkeypatch, tmp_path):
    """build() with compiling and linking replaced by a list of what was linked."""
    linked = []
    monkeypatch.setattr(build, "_compile", lambda src, poison=False: f"{src}{poison}")
    monkeypatch.setattr(build, "_link", lambda objs, out: linked.append(out))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    return linked


def no_compiler(*args, **kw):
    raise FileNotFoundError("g++")


def test_without_a_host_compiler(traced, monkeypatch, tmp_path):
    (tmp_path / "_marshal.so").write_text("of an older build")
    monkeypatch.setattr(subprocess, "run", no_compiler)
    with pytest.warns(UserWarning, match="ctypes"):
        assert build.build() == build.LIB
    assert traced == [build.LIB, build.POISON_LIB]
    assert not (tmp_path / "_marshal.so").exists()


def test_a_failed_library_is_still_an_error(traced, monkeypatch):
    monkeypatch.setattr(build, "_build_marshal", lambda: None)

    def fails(src, poison=False):
        raise RuntimeError("hipcc failed")

    monkeypatch.setattr(build, "_compile", fails)
    with pytest.raises(RuntimeError, match="hipcc"):
        build.build()
    assert traced == []


def test_with_everything(traced, monkeypatch, recwarn):
    monkeypatch.setattr(build, "_build_marshal", lambda: None)
    assert build.build() == build.LIB
    assert traced == [build.LIB, build.POISON_LIB] and not recwarn
