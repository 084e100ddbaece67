"""Build the CUDA library ``libqmm.so`` in-tree with nvcc, for sm_103a only.

Each translation unit under ``csrc/`` is compiled in parallel to an object in
``_build/`` and the objects are linked into ``libqmm.so`` next to this file,
with the CUDA runtime linked statically so the library loads on a host that
has the toolkit but no driver (the exported-symbol checks run there). The
host-only ``csrc/binding.cpp`` becomes the Python module ``_binding`` (argument
marshalling against torch's headers), linked to ``libqmm.so``.
A rebuild happens only when a source or header is newer than the library made of it,
or, of ``_binding``, when Python or torch is another one than it was built for.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libqmm.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(PKG_DIR, "_binding.so")
BINDING_TAG = os.path.join(PKG_DIR, "_binding.tag")   # beside it: what it was built for
HEADERS = [os.path.join(REPO_DIR, "include", "qmm.h")]

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "-I" + os.path.join(REPO_DIR, "include")]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqmm.so")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newer(inputs: list[str], path: str) -> bool:
    """path is missing or older than one of the inputs."""
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in inputs)


def library_stale() -> bool:
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return _newer(sources() + hdrs + HEADERS + [__file__], LIB_PATH)


def binding_stale() -> bool:
    if _newer(HEADERS + [BINDING_SRC, __file__], BINDING_PATH) or not os.path.exists(BINDING_TAG):
        return True
    with open(BINDING_TAG) as f:
        return f.read() != binding_tag()


def needs_build() -> bool:
    return library_stale() or binding_stale()


def binding_tag() -> str:
    """The Python and the torch that a _binding built now is for: their binary interfaces
    differ from version to version."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{_torch_dir()}\n{f.read()}"


def _torch_dir() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _cxx() -> str:
    return os.environ.get("CXX") or shutil.which("g++") or "c++"


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
    if src == BINDING_SRC:
        cuda = os.path.dirname(os.path.dirname(nvcc_path()))
        cmd = [_cxx(), "-O2", "-std=c++17", "-fPIC", "-Wall", "-I" + os.path.join(_torch_dir(), "include"),
               "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"), "-c", src, "-o", obj]
    else:
        cmd = [nvcc_path(), *ARCH_FLAGS, *NVCC_FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {os.path.basename(src)} failed:\n{r.stdout}\n{r.stderr}")
    return obj


def _link(cmd: list[str], path: str) -> None:
    tmp = path + ".tmp"
    r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {os.path.basename(path)} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def _make(library: bool, binding: bool) -> None:
    """Compile and link the two, each if asked for."""
    if not library and not binding:
        return
    tlib = os.path.join(_torch_dir(), "lib")
    if binding and not os.path.exists(os.path.join(tlib, "libtorch_cuda.so")):
        raise RuntimeError("this torch has no CUDA libraries to link _binding to")
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = ([BINDING_SRC] if binding else []) + (sources() if library else [])
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(_compile, srcs))
    bobj = objs.pop(0) if binding else None
    if library:
        _link([nvcc_path(), *ARCH_FLAGS, "-shared", "-cudart", "static", *objs], LIB_PATH)
    if binding:
        _link([_cxx(), "-shared", bobj, "-L" + PKG_DIR, "-l:libqmm.so", "-Wl,-rpath,$ORIGIN", "-L" + tlib,
               "-Wl,-rpath," + tlib, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"],
              BINDING_PATH)
        with open(BINDING_TAG, "w") as f:
            f.write(binding_tag())


def build_library() -> str:
    """Compile and link libqmm.so if needed; return its path."""
    _make(library_stale(), False)
    return LIB_PATH


def build_binding() -> None:
    """Compile and link _binding.so if needed (libqmm.so is there)."""
    _make(False, binding_stale())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link both if needed; return libqmm.so's path."""
    _make(force or library_stale(), force or binding_stale())
    if verbose:
        print(f"built {LIB_PATH}")
    return LIB_PATH


if __name__ == "__main__":
    build(force=True, verbose=True)
