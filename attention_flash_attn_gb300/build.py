"""Builds libattn_gb300.so in-tree from csrc/*.cu with nvcc for sm_103a.

Every translation unit is compiled in parallel (one nvcc process each) into ``_build/``
and linked into ``attention_flash_attn_gb300/libattn_gb300.so`` with the CUDA runtime
linked statically, so the library loads without a GPU or a driver (the driver entry
points it needs are resolved at run time).  csrc/binding.cpp, the calls that cache.py makes, is
compiled with g++ against PyTorch's headers into ``_binding.so`` beside it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libattn_gb300.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
         "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _hash(files, *words) -> str:
    h = hashlib.sha256()
    for f in files:
        h.update(os.path.relpath(f, ROOT).encode())  # relative: the same sources hash alike anywhere
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(words).encode())
    return h.hexdigest()


def _headers():
    return sorted(glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stamp() -> str:
    """Of the library: its sources and flags."""
    own = sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")))
    return _hash(_sources() + own + _headers(), *ARCH, *FLAGS)


def _binding_stamp() -> str:
    """Of the binding: its source, the PyTorch and the Python that it is compiled for."""
    return _hash([BINDING_SRC] + _headers(), torch.__version__, sys.version)


def _current(path: str, stamp_file: str, stamp: str) -> bool:
    if not os.path.exists(path) or not os.path.exists(stamp_file):
        return False
    with open(stamp_file) as fh:
        return fh.read() == stamp


def _write(path: str, text: str) -> None:
    with open(path, "w") as fh:
        fh.write(text)


# Sources that the backward main kernel's code depends on: a DRAM-traffic figure recorded by
# ncu for that kernel stays valid while these files (and the flags) are unchanged.
BWD_MAIN_SOURCES = ("bwd_tc.cu", "bwd_score.cuh", "tc_common.cuh", "tc_host.cu", "common.cuh", "internal.h")


def _code_only(text: str) -> str:
    """C / C++ source with comments and whitespace removed (string literals kept), so that an
    edit to comments alone leaves a kernel's stamp unchanged."""
    out, i, n = [], 0, len(text)
    while i < n:
        c = text[i]
        if c == '"' or c == "'":
            j = i + 1
            while j < n and text[j] != c:
                j += 2 if text[j] == "\\" else 1
            out.append(text[i:j + 1])
            i = j + 1
        elif text.startswith("//", i):
            i = text.find("\n", i)
            i = n if i < 0 else i
        elif text.startswith("/*", i):
            j = text.find("*/", i + 2)
            i = n if j < 0 else j + 2
        else:
            if not c.isspace():
                out.append(c)
            i += 1
    return "".join(out)


def kernel_stamp(names=BWD_MAIN_SOURCES) -> str:
    """Hash of the code (comments and whitespace removed) of the named csrc files and the
    public header, and of the compile flags."""
    h = hashlib.sha256()
    files = [os.path.join(CSRC, n) for n in names] + [os.path.join(ROOT, "include", "attn_gb300.h")]
    for f in files:
        h.update(os.path.relpath(f, ROOT).encode())
        with open(f, encoding="utf-8") as fh:
            h.update(_code_only(fh.read()).encode())
    h.update(" ".join(ARCH + FLAGS).encode())
    return h.hexdigest()


def _compile_binding(out: str) -> None:
    """g++ of csrc/binding.cpp against the PyTorch that runs this (its headers' directory, its libraries)."""
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for i in inc for x in ("-isystem", i)], BINDING_SRC, "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")


def _link_binding(obj: str) -> None:
    tmp = BINDING + f".tmp{os.getpid()}"
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libattn_gb300.so", "-Wl,-rpath,$ORIGIN", "-L", lib, "-ltorch_python",
           "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what has changed and return the path of the shared library.  The library needs nvcc alone; it is linked
    before a failure of the binding's compilation (which needs PyTorch's headers) is raised."""
    os.makedirs(BUILD, exist_ok=True)
    lib_stamp, binding_stamp = (os.path.join(BUILD, n) for n in ("stamp", "stamp_binding"))
    make_lib = force or not _current(LIB, lib_stamp, _stamp())
    make_binding = force or not _current(BINDING, binding_stamp, _binding_stamp())
    binding_obj = os.path.join(BUILD, "binding.o")
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(_compile_binding, binding_obj) if make_binding else None
        if make_lib:
            _build_lib(ex, srcs, verbose)
            _write(lib_stamp, _stamp())
        if binding:
            binding.result()
    if make_binding:
        _link_binding(binding_obj)
        _write(binding_stamp, _binding_stamp())
    return LIB


def _build_lib(ex, srcs, verbose: bool) -> None:
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    results = list(ex.map(compile_one, srcs))
    log = "\n".join(err for _, err in results)
    _write(os.path.join(BUILD, "ptxas.log"), log)
    if verbose:
        print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "--cudart", "static", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force=True, verbose=True))
