"""Building: the library needs no Python headers, the Python extension belongs
to one interpreter (no GPU needed)."""

import os
import subprocess
import sys
import sysconfig

import pytest

lm = pytest.importorskip("layout_driven_movement_gb300")
from layout_driven_movement_gb300 import _build  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    lm.lib()


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The extension goes to a place of its own and is not loaded yet."""
    monkeypatch.setattr(_build, "PYCALL", str(tmp_path / "_pycall.so"))
    monkeypatch.setattr(_build, "PYCALL_LOG", str(tmp_path / "pycall.log"))
    monkeypatch.setattr(lm, "_pycall_module", None)
    return tmp_path


def test_the_library_builds_without_python_headers(elsewhere, monkeypatch,
                                                   capfd):
    (elsewhere / "_pycall.so").write_bytes(b"of an earlier build")
    os.utime(elsewhere / "_pycall.so", (0, 0))
    monkeypatch.setattr(_build.sysconfig, "get_path",
                        lambda name: str(elsewhere / "no headers"))
    assert _build.build() == _build.LIB
    assert "Python.h" in capfd.readouterr().err
    # nothing stale is left to be loaded, and the calls say what is missing
    assert not os.path.exists(_build.PYCALL)
    with pytest.raises(RuntimeError, match="Python.h"):
        lm._pycall()
    # plans need the library only
    assert lm.RopePlan(64).rotary_dim == 64


def test_the_extension_without_a_compiler(elsewhere, monkeypatch):
    monkeypatch.setenv("CC", str(elsewhere / "no compiler"))
    assert _build.build() == _build.LIB
    with pytest.raises(RuntimeError, match="no compiler"):
        lm._pycall()


def test_the_extension_is_the_interpreters_own():
    assert os.path.basename(_build.PYCALL) == \
        "_pycall" + sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.exists(_build.PYCALL)
    assert lm._pycall().__file__ == _build.PYCALL


def test_the_extension_is_linked_again_when_the_library_is_newer():
    os.utime(_build.PYCALL, (0, 0))
    _build.build()
    assert os.path.getmtime(_build.PYCALL) >= os.path.getmtime(_build.LIB)


def test_a_moved_tree_uses_its_own_library(tmp_path):
    """The extension names the library beside it, not the place where it was
    built: a copy of the package works where the first one is still there, and
    loads the library once."""
    import shutil
    place = tmp_path / "layout_driven_movement_gb300"
    shutil.copytree(_build.PKG, place,
                    ignore=shutil.ignore_patterns("_build", "__pycache__"))
    code = ("import layout_driven_movement_gb300 as lm\n"
            "lm.lib(); lm._pycall()\n"
            "print(*sorted({l.split()[-1] for l in open('/proc/self/maps')\n"
            "               if 'liblayoutmove' in l or '_pycall' in l}),\n"
            "      sep='\\n')\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=tmp_path,
                         env={**os.environ, "PYTHONPATH": str(tmp_path)},
                         capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split() == sorted(
        str(place / os.path.basename(f)) for f in (_build.LIB, _build.PYCALL))
