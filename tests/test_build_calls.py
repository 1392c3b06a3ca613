"""The build of the short way from Python to the 8-bit layer's calls, which is optional: without it
ctypes makes the same calls."""
import os
import subprocess
import sys

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


def test_extension_is_rebuilt_by_itself(paths, monkeypatch):
    """Older than its source or the C header, the extension is built again although the library is fresh."""
    build.build()
    assert os.path.exists(build.CALLS)
    fresh = os.path.getmtime(build.CALLS)
    build.build()
    assert os.path.getmtime(build.CALLS) == fresh
    for dep in (build.CALLS_SRC, build.HEADER):
        before = os.path.getmtime(dep) - 10
        os.utime(build.CALLS, (before, before))
        lib = os.path.getmtime(build.LIB)
        build.build()
        assert os.path.getmtime(build.CALLS) > before and os.path.getmtime(build.LIB) == lib


@pytest.mark.parametrize("flags,used", [([], False), (["-DS2_HEADER_ID=another"], False), (None, True)])
def test_only_an_extension_of_the_same_header_is_used(tmp_path, flags, used):
    """One that was compiled from another header would pass its arguments under other signatures:
    ctypes makes the calls then."""
    calls = str(tmp_path / "_s2calls.so")
    subprocess.run([os.environ.get("CXX") or "g++", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", build._python_headers(), "-I",
                    os.path.dirname(build.HEADER), *(build.header_flags() if flags is None else flags), build.CALLS_SRC, "-o", calls],
                   check=True)
    code = ("import ctypes, sketch_compressed_sparse_gb300 as s2\n"
            f"s2._CALLS_PATH = {calls!r}\n"
            "kinds = [isinstance(s2._f(n), ctypes._CFuncPtr) for n in ('s2_pack8', 's2_unpack8', 's2_matmul8', 's2_wgrad8')]\n"
            f"assert kinds == [{not used}] * 4, kinds\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=build.ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
