"""Host-side tests of the build's rules: what the Python module needs beside
the C library, and when it is built again. Nothing is compiled here."""
import os

import pytest

from row_wise_normalization_rmsnorm_gb300 import build as rn_build


def refuse(*a, **k):
    raise AssertionError("nothing is to be compiled")


@pytest.fixture
def up_to_date(monkeypatch, tmp_path):
    """A library and a module that nothing has changed for; the paths of the
    module and its stamp."""
    rn_build.build()
    ext, stamp = tmp_path / "_heads_ext.so", tmp_path / "stamp"
    ext.write_bytes(b"")
    stamp.write_text(rn_build._ext_for(), encoding="utf-8")
    monkeypatch.setattr(rn_build, "EXT", str(ext))
    monkeypatch.setattr(rn_build, "EXT_STAMP", str(stamp))
    monkeypatch.setattr(rn_build, "_compile", refuse)
    monkeypatch.setattr(rn_build, "_compile_ext", refuse)
    return ext, stamp


def test_nothing_changed_builds_nothing(up_to_date):
    assert not rn_build._ext_stale(False)
    assert rn_build.build() == rn_build.LIB


def test_another_pytorch_or_python_makes_the_module_stale(up_to_date):
    ext, stamp = up_to_date
    stamp.write_text(rn_build._ext_for().replace("__version__", "__version_of_another__"), encoding="utf-8")
    assert rn_build._ext_stale(False)
    stamp.unlink()
    assert rn_build._ext_stale(False)


@pytest.mark.parametrize("lacks", ["torch", "headers", "python", "compiler"])
def test_the_library_needs_none_of_what_the_module_does(up_to_date, monkeypatch, tmp_path, capsys, lacks):
    ext, stamp = up_to_date
    stamp.write_text("another", encoding="utf-8")
    if lacks == "torch":
        def none():
            raise RuntimeError("PyTorch is required to build the Python module")
        monkeypatch.setattr(rn_build, "_torch_dir", none)
        what = "PyTorch"
    elif lacks == "headers":
        monkeypatch.setattr(rn_build, "_torch_dir", lambda: str(tmp_path))
        what = "headers"
    elif lacks == "python":
        monkeypatch.setattr(rn_build, "_python_include", lambda: str(tmp_path))
        what = "Python.h"
    else:
        monkeypatch.setattr(rn_build.shutil, "which", lambda name: None)
        what = "g++"
    assert rn_build.build() == rn_build.LIB
    assert what in capsys.readouterr().err
    assert not os.path.exists(ext)  # a stale module is not left to be loaded


def test_everything_is_here():
    assert rn_build._ext_missing() is None
