"""A native module built for another Python or PyTorch is rebuilt, and until then
its import says so; the command that the errors name works without the package."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(tmp_path, monkeypatch):
    from tests.conftest import build_library
    build_library()
    import __graft_entry__
    mod = __graft_entry__._build_module()
    monkeypatch.setattr(mod, "BUILT_FOR", str(tmp_path / "native_for.txt"))
    return mod


def _write(path, text):
    with open(path, "w") as f:
        f.write(text)


def test_another_version_is_out_of_date(build):
    assert build.built_for() == "" and not build.up_to_date()
    _write(build.BUILT_FOR, build.versions())
    assert build.up_to_date()
    _write(build.BUILT_FOR, build.versions() + ".1")
    assert not build.up_to_date()


def test_import_names_the_versions(monkeypatch, build):
    from linear_cross_entropy_gb300 import _lib
    _write(build.BUILT_FOR, "cpython-37, torch 1.0")
    monkeypatch.setattr(_lib, "_lib", None)
    monkeypatch.setattr(_lib.build, "BUILT_FOR", build.BUILT_FOR)
    with pytest.raises(ImportError, match="torch 1.0.*build.py"):
        _lib.load()
    _write(build.BUILT_FOR, build.versions())
    assert _lib.load() is not None


def test_the_command_runs_without_a_built_package(tmp_path, build):
    """In a tree with the sources and nothing built, as far as the compiler."""
    shutil.copytree(os.path.join(ROOT, "linear_cross_entropy_gb300"), tmp_path / "linear_cross_entropy_gb300",
                    ignore=shutil.ignore_patterns("*.so", "_build", "__pycache__"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    env = {**os.environ, "PATH": ""}  # no compiler: the build itself is not repeated
    words = build.COMMAND.split()
    assert words[0] == "python"
    r = subprocess.run([sys.executable] + words[1:], cwd=tmp_path, env=env, capture_output=True, text=True)
    assert "ImportError" not in r.stderr and "nvcc" in r.stderr, r.stderr
