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
Python binding's fast path, where torch is installed: into ``_binding.*.so``,
whose name holds the versions that it fits.
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
SOURCES = [os.path.join(CSRC, f) for f in ("mla_decode.cu", "mla_kv_pack.cu", "mla_sparse.cu", "mla_cascade.cu",
                                               "mla_chunk.cu", "mla_mass.cu", "mla_evict.cu", "mla_tree.cu", "mla_verify.cu",
                                               "mla_pages.cu", "mla_rope.cu")]
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _headers():
    return [os.path.join(d, f) for d in (CSRC, INCLUDE) for f in os.listdir(d) if f.endswith((".cuh", ".h"))]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build the library")


def _newer(path: str, sources) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in sources)


def _have_torch() -> bool:
    try:
        import torch  # noqa: F401
    except Exception:  # not there, or its libraries do not load
        return False
    return True


def up_to_date() -> bool:
    """The library and, where there is a torch to load it, the binding."""
    return _newer(LIB_PATH, [*SOURCES, *_headers()]) and (not _have_torch() or _binding_up_to_date())


def binding_path() -> str:
    """Where the binding for this interpreter and this torch is.  It reads
    their objects' layouts, which differ between releases, so the name holds
    both: a module built for others is not this one."""
    import sysconfig

    import torch

    cxx11 = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(PKG, f"_binding.torch-{torch.__version__}-abi{cxx11}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _binding_up_to_date() -> bool:
    return _newer(binding_path(), [BINDING_SOURCE, *_headers()])


def _run(what, cmd):
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"{what} failed: {e}") from e
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    return res.stdout + res.stderr


def _build_library(verbose: bool) -> None:
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [
        nvcc_path(), "-shared", "-Xcompiler", "-fPIC", *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17",
        "-I", INCLUDE, "-I", CSRC, "-cudart", "shared", "--threads", "0", "-o", tmp, *SOURCES,
    ]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    try:
        out = _run("nvcc", cmd)
        if verbose:
            sys.stderr.write(out)
        os.replace(tmp, LIB_PATH)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)


def _compile_binding(obj: str) -> None:
    import sysconfig

    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")
    _run("compiling the binding",
         ["g++", "-c", "-O2", "-fPIC", "-std=c++17", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", inc, "-I", sysconfig.get_paths()["include"], "-I", cuda, "-I", INCLUDE, BINDING_SOURCE, "-o", obj])


def _link_binding(obj: str, tmp: str) -> None:
    import torch

    _run("linking the binding",
         ["g++", "-shared", obj, "-o", tmp, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python",
          "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L", PKG, f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, binding_path())


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile the shared library and the binding in place; returns the
    library's path.  The library needs nvcc alone and is there whatever becomes
    of the binding, which needs torch and its headers: without torch it is left
    out, and an error in it is raised once the library is in place."""
    if not force and up_to_date():
        return LIB_PATH
    from concurrent.futures import ThreadPoolExecutor

    obj, tmp = (os.path.join(PKG, f"_binding.tmp{os.getpid()}{end}") for end in (".o", ".so"))
    with ThreadPoolExecutor(1) as beside:
        binding = beside.submit(_compile_binding, obj) if _have_torch() else None
        try:
            if force or not _newer(LIB_PATH, [*SOURCES, *_headers()]):
                _build_library(verbose)
            if binding is None:
                sys.stderr.write("torch is not importable: the library is built, its Python binding is not\n")
            else:
                binding.result()
                _link_binding(obj, tmp)
        finally:
            if binding is not None:
                binding.exception()  # (ends before its output is removed)
            for f in (obj, tmp):
                if os.path.exists(f):
                    os.remove(f)
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
