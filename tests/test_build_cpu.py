"""The in-tree build without a GPU: what of the library and the binding is there
when one of the two cannot be built.  (Compilers are stand-ins that write a
file, in a folder of the test's.)"""
import os
import subprocess
import sys

import pytest

from paged_mla_decode_09_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def tool(path, body):
    path.write_text("#!/bin/sh\n" + body)
    path.chmod(0o755)
    return str(path)


WRITES = 'while [ "$1" != -o ]; do shift; done; echo built > "$2"\n'


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build.py with outputs in tmp_path, an nvcc that works, and the given g++."""
    (tmp_path / "bin").mkdir()
    monkeypatch.setenv("NVCC", tool(tmp_path / "bin" / "nvcc", WRITES))
    monkeypatch.setenv("PATH", f"{tmp_path}/bin:/usr/bin:/bin")
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libmla_decode.so"))
    monkeypatch.setattr(build, "binding_path", lambda: str(tmp_path / "_binding.so"))
    tool(tmp_path / "bin" / "g++", WRITES)
    return tmp_path


def left(tree):
    return sorted(f for f in os.listdir(tree) if f != "bin")


def test_both(tree):
    pytest.importorskip("torch")
    assert not build.up_to_date()
    assert build.build_library() == build.LIB_PATH
    assert left(tree) == ["_binding.so", "libmla_decode.so"] and build.up_to_date()


@pytest.mark.parametrize("gxx", ["echo no such header; exit 1\n", None])
def test_a_binding_that_does_not_compile_leaves_the_library(tree, monkeypatch, gxx):
    pytest.importorskip("torch")
    if gxx is None:
        os.remove(tree / "bin" / "g++")
        monkeypatch.setenv("PATH", f"{tree}/bin")
    else:
        tool(tree / "bin" / "g++", gxx)
    with pytest.raises(RuntimeError, match="binding"):
        build.build_library()
    assert left(tree) == ["libmla_decode.so"]
    before = os.stat(build.LIB_PATH).st_mtime_ns
    tool(tree / "bin" / "g++", WRITES)  # mended: the library is not built again
    monkeypatch.setenv("PATH", f"{tree}/bin:/usr/bin:/bin")
    build.build_library()
    assert left(tree) == ["_binding.so", "libmla_decode.so"] and os.stat(build.LIB_PATH).st_mtime_ns == before


def test_a_library_that_does_not_compile_leaves_nothing(tree):
    tool(tree / "bin" / "nvcc", "echo no; exit 2\n")
    with pytest.raises(RuntimeError, match="nvcc"):
        build.build_library()
    assert left(tree) == []


@pytest.mark.parametrize("torch", ["", "raise OSError('libcudart.so: cannot open shared object file')"])
def test_without_torch_there_is_the_library(tree, torch):
    (tree / "bin" / "torch").mkdir()
    (tree / "bin" / "torch" / "__init__.py").write_text(torch)
    code = f"""
import sys
sys.path[:0] = [{ROOT!r}, {str(tree / "bin")!r}]
if not {torch!r}:
    sys.modules["torch"] = None  # not there: an import raises ImportError
from paged_mla_decode_09_gb300 import build
build.LIB_PATH = {build.LIB_PATH!r}
assert not build.up_to_date()
assert build.build_library() == build.LIB_PATH and build.up_to_date()
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert "binding is not" in r.stderr and left(tree) == ["libmla_decode.so"]


def test_a_binding_of_another_torch_or_python_is_another_file(monkeypatch):
    """It would read tensors by the wrong layout: it is neither up to date nor loaded."""
    import sysconfig

    torch = pytest.importorskip("torch")
    import paged_mla_decode_09_gb300 as mla

    build.build_library()
    here = build.binding_path()
    assert os.path.exists(here) and build.up_to_date()
    monkeypatch.setattr(mla, "_fast", None)
    assert mla._binding() is mla._binding()
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    real = sysconfig.get_config_var
    for patch in ((torch, "__version__", "9.9.9+cu999"), (torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI),
                  (sysconfig, "get_config_var", lambda k: suffix.replace("cpython-3", "cpython-9") if k == "EXT_SUFFIX" else real(k))):
        with monkeypatch.context() as m:
            m.setattr(*patch)
            m.setattr(mla, "_fast", None)
            assert build.binding_path() != here and not build.up_to_date()
            with pytest.raises(RuntimeError, match="missing"):
                mla._binding()
    assert build.binding_path() == here and build.up_to_date()
