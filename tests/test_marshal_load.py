"""CPU: the binding without its compiled short way, or with one that does not fit:
a warning at the first call, and every call goes through ctypes."""
import sys
import types
import warnings

import pytest

import fp8_fine_grained_fp8bs_amd as package
from fp8_fine_grained_fp8bs_amd import fp8bs
from tests.test_marshal import NAMES, arguments


@pytest.fixture(autouse=True)
def unloaded(monkeypatch, tmp_path):
    path = tmp_path / "_marshal.so"
    path.write_text("a file")
    monkeypatch.setattr(fp8bs, "_marshal", None)
    monkeypatch.setattr(fp8bs, "MARSHAL_PATH", str(path), raising=False)
    monkeypatch.delattr(package, "_marshal", raising=False)
    return path


def calls_go_through_ctypes():
    for name in NAMES:
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            assert fp8bs._short(name, *arguments("cpu", name)) is None


def test_missing(unloaded):
    unloaded.unlink()
    calls_go_through_ctypes()


def test_unloadable(monkeypatch):
    monkeypatch.setitem(sys.modules, package.__name__ + "._marshal", None)   # its import raises
    with pytest.warns(UserWarning, match="ctypes"):
        assert fp8bs._short(NAMES[0], *arguments("cpu", NAMES[0])) is None
    calls_go_through_ctypes()


@pytest.mark.parametrize("version", ["0.0", None])
def test_built_for_another_torch(monkeypatch, version):
    """Its functions are not called: they look into torch's objects."""
    def never(*args):
        raise AssertionError("called")

    module = types.SimpleNamespace(**{n[6:]: never for n in NAMES})
    if version is not None:
        module.torch_version = version
    monkeypatch.setitem(sys.modules, package.__name__ + "._marshal", module)
    with pytest.warns(UserWarning, match="ctypes"):
        assert fp8bs._short(NAMES[0], *arguments("cpu", NAMES[0])) is None
    calls_go_through_ctypes()
