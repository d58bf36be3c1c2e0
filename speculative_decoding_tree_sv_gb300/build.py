"""Build ``lib/libsv.so`` in-tree with nvcc for sm_103a.

Each CUDA translation unit is compiled in parallel, then linked into one
shared library with the CUDA runtime linked statically (the library loads on
machines without a GPU driver; the driver is resolved at first use).  Where
torch is installed, the Python module that checks and passes the cache
operators' tensors goes beside it.  That module reads torch's own objects, so it
is compiled against the installed torch's headers and its file name carries the
torch and Python it was built for: another pair builds its own.
"""

from __future__ import annotations

import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
LIBDIR = os.path.join(PKG, "lib")
LIBNAME = "libsv.so"
SOURCES = ["abi.cu", "tree_attention.cu", "tree_attention_wide.cu", "tree_attention_dealt.cu", "greedy_accept.cu",
           "sample_accept.cu", "kv_commit.cu", "retrieval.cu", "kv_append.cu", "rope_append.cu", "sample_tokens.cu", "pages.cu",
           "chunk_attention.cu", "chunk_rows.cu", "chunk_tiles.cu", "prefix_attention.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the sv library needs the CUDA toolkit to build")


def library_path() -> str:
    return os.path.join(LIBDIR, LIBNAME)


def _torch_dir() -> Optional[str]:
    """Where torch is installed; None without it."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    return spec.submodule_search_locations[0]


def _torch_version(torch_dir: str) -> str:
    with open(os.path.join(torch_dir, "version.py")) as f:
        found = re.search(r"^__version__\s*(?::[^=]*)?=\s*['\"]([^'\"]+)", f.read(), re.M)
    if found is None:
        raise RuntimeError(f"no __version__ in {torch_dir}/version.py")
    return found.group(1)


def marshal_path() -> Optional[str]:
    """The tensor module of this Python and the installed torch; None without torch."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return None
    return os.path.join(LIBDIR, f"_marshal-torch{_torch_version(torch_dir)}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "sv.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    built = [f for f in (library_path(), marshal_path()) if f is not None]
    if not all(os.path.exists(f) for f in built):
        return False
    t = min(os.path.getmtime(f) for f in built)
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    lib = library_path()
    if not force and up_to_date():
        return lib
    os.makedirs(LIBDIR, exist_ok=True)
    objdir = os.path.join(LIBDIR, "obj")
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                    "--expt-relaxed-constexpr"]
    if ptxas_info:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(objdir, os.path.splitext(src)[0] + ".o")
        cmd = [cc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj, r.stderr

    module = marshal_path()

    def compile_marshal():
        if module is None:
            return None
        obj = os.path.join(objdir, "marshal.o")
        torch_dir = _torch_dir()
        include = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                   sysconfig.get_paths()["include"]]
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, "marshal.cpp"), "-o", obj]
        for path in include:
            cmd += ["-isystem", path]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for marshal.cpp:\n{r.stderr}")
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        marshal = ex.submit(compile_marshal)
        results = list(ex.map(compile_one, SOURCES))
    if verbose or ptxas_info:
        for (_, err), src in zip(results, SOURCES):
            if err.strip():
                sys.stderr.write(f"--- {src}\n{err}")
    tmp = lib + ".tmp"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    module_obj = marshal.result()  # (the library is in place, whatever became of it)
    if module_obj is None:
        if verbose:
            sys.stderr.write("torch is not installed: built without the tensor module\n")
        return lib
    tmp = module + ".tmp"
    # torch's libraries are in the process by the time the module is loaded
    cmd = ["g++", "-shared", "-o", tmp, module_obj, "-L", LIBDIR, "-l:" + LIBNAME, "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(module)} failed:\n{r.stderr}")
    os.replace(tmp, module)
    return lib


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(library_path())
