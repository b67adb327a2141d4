"""In-tree build of the CUDA library (sm_103a only).

``python -m paged_mla_decode_09_gb300.build`` compiles
``csrc/mla_decode.cu`` (the decode), ``csrc/mla_kv_pack.cu`` (the cache
write), ``csrc/mla_sparse.cu`` (the top-k decode), ``csrc/mla_cascade.cu``
(the shared-prefix cascade), ``csrc/mla_chunk.cu`` (prompt chunks and
windows), ``csrc/mla_mass.cu`` (attention mass), ``csrc/mla_evict.cu``
(eviction), ``csrc/mla_tree.cu`` (trees of drafts), ``csrc/mla_verify.cu``
(their verification), ``csrc/mla_pages.cu`` (page operations) and
``csrc/mla_rope.cu`` (rotary cache write) with nvcc into
``libmla_decode.so`` next to this file.  One ``-gencode``, the files in
parallel; a few seconds.  Beside it g++ compiles ``csrc/binding.cpp``, the
Python binding's fast path, into ``_binding.so``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libmla_decode.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(PKG, "_binding.so")
SOURCES = [os.path.join(CSRC, f) for f in ("mla_decode.cu", "mla_kv_pack.cu", "mla_sparse.cu", "mla_cascade.cu",
                                               "mla_chunk.cu", "mla_mass.cu", "mla_evict.cu", "mla_tree.cu", "mla_verify.cu",
                                               "mla_pages.cu", "mla_rope.cu")]
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def depends():
    files = [*SOURCES, BINDING_SOURCE]
    for d in (CSRC, INCLUDE):
        files += [os.path.join(d, f) for f in os.listdir(d) if f.endswith((".cuh", ".h"))]
    return files


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build the library")


def up_to_date() -> bool:
    if not (os.path.exists(LIB_PATH) and os.path.exists(BINDING_PATH)):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    return all(os.path.getmtime(p) <= t for p in depends())


def _failed(what, cmd, out):
    return RuntimeError(f"{what} failed:\n" + " ".join(cmd) + "\n" + out)


def _compile_binding(obj: str):
    """g++ on the binding's source, started; returns (process, command)."""
    import sysconfig

    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")
    cmd = ["g++", "-c", "-O2", "-fPIC", "-std=c++17", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", inc, "-I", sysconfig.get_paths()["include"], "-I", cuda, "-I", INCLUDE, BINDING_SOURCE, "-o", obj]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True), cmd


def _link_binding(obj: str, tmp: str):
    import torch

    cmd = ["g++", "-shared", obj, "-o", tmp, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L", PKG, f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise _failed("linking the binding", cmd, res.stdout + res.stderr)
    os.replace(tmp, BINDING_PATH)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile the shared library and the binding in place; returns the library's path."""
    if not force and up_to_date():
        return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    obj = BINDING_PATH + f".tmp{os.getpid()}.o"
    cmd = [
        nvcc_path(), "-shared", "-Xcompiler", "-fPIC", *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17",
        "-I", INCLUDE, "-I", CSRC, "-cudart", "shared", "--threads", "0", "-o", tmp, *SOURCES,
    ]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    binding, binding_cmd = _compile_binding(obj)
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
        out, _ = binding.communicate()
        if res.returncode != 0:
            raise _failed("nvcc", cmd, res.stdout + res.stderr)
        if verbose:
            sys.stderr.write(res.stdout + res.stderr)
        if binding.returncode != 0:
            raise _failed("compiling the binding", binding_cmd, out)
        os.replace(tmp, LIB_PATH)
        _link_binding(obj, BINDING_PATH + f".tmp{os.getpid()}")
    finally:
        for f in (tmp, obj):
            if os.path.exists(f):
                os.remove(f)
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
