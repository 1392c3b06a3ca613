"""The build of the short way from Python to the 8-bit layer's calls, which is optional: without it
ctypes makes the same calls."""
import os

import pytest

from sketch_compressed_sparse_gb300 import build

pytestmark = pytest.mark.skipif(build._python_headers() is None, reason="no Python headers")


@pytest.fixture
def paths(tmp_path, monkeypatch):
    """The extension's paths, away from the real ones."""
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_s2calls.so"))
    monkeypatch.setattr(build, "LIBDIR", str(tmp_path))
    return tmp_path


@pytest.mark.parametrize("cxx", ["/nowhere/g++", "false"])
def test_build_goes_on_without_a_host_compiler(paths, monkeypatch, capsys, cxx):
    """Nothing is raised, the reason is printed, and an extension of an earlier build does not stay."""
    with open(build.CALLS, "w") as f:
        f.write("old")
    monkeypatch.setenv("CXX", cxx)
    build._build_calls()
    assert not os.path.exists(build.CALLS)
    assert "_s2calls" in capsys.readouterr().err
    assert os.listdir(paths) == []
