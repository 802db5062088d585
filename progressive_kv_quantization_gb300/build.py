"""Builds the in-tree CUDA library ``_build/liblynx.so`` for sm_103a with nvcc,
and ``_build/lynx_binding.so``, the native part of the Python binding.

Each .cu file compiles to an object in parallel; the objects link into one
shared library with the CUDA runtime linked statically, so the library needs
only the NVIDIA driver at run time.  The binding (one C++ file against torch's
headers) links to that library; where it cannot be built (no torch, no g++) the
library is there all the same and a warning says what is missing.  Each is built
again when one of its sources or headers is newer, the binding also for another
torch or Python.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor
from importlib import metadata

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "liblynx.so")
BINDING = os.path.join(BUILD, "lynx_binding.so")

SOURCES = ["lynx_api.cu", "encode.cu", "reconstruct.cu", "decode_attn.cu", "decode_quant.cu", "decode_tc.cu",
           "decode_narrow.cu", "decode_draft.cu", "decode_bf16.cu",
           "decode_noalloc.cu", "assign_pages.cu", "qkv_append.cu", "verify_drafts.cu",
           "chunk_attn.cu", "decode_e4m3.cu", "token_logprobs.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the Lynx CUDA library cannot be built")
    return exe


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files.append(os.path.join(INCLUDE, "lynx.h"))
    return files


def _newer(target: str, files) -> bool:
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in files)


def up_to_date() -> bool:
    return os.path.exists(LIB) and _newer(LIB, _inputs())


def _binding_of() -> str:
    """The torch and Python that the binding is built for."""
    try:
        return f"torch {metadata.version('torch')} {sysconfig.get_config_var('SOABI')}"
    except metadata.PackageNotFoundError:
        return "no torch"


def binding_up_to_date() -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING + ".of"):
        return False
    with open(BINDING + ".of") as f:
        of = f.read()
    return of == _binding_of() and _newer(BINDING, [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "lynx.h")])


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile (if needed) and return the path of liblynx.so."""
    library, binding = force or not up_to_date(), force or not binding_up_to_date()
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    def compile_binding():
        import torch   # its headers
        inc = os.path.join(os.path.dirname(torch.__file__), "include")
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")
        obj = os.path.join(BUILD, "binding.o")
        dirs = [INCLUDE, sysconfig.get_paths()["include"], inc, os.path.join(inc, "torch", "csrc", "api", "include"), cuda]
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *[f"-I{d}" for d in dirs], "-c",
               os.path.join(CSRC, "binding.cpp"), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
        return obj, os.path.join(os.path.dirname(torch.__file__), "lib")

    def link(what, tmp, target, cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"linking {what} failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, target)

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        made = ex.submit(compile_binding) if binding else None
        objs = list(ex.map(compile_one, SOURCES)) if library else []
    if library:
        tmp = LIB + ".tmp"
        link("liblynx.so", tmp, LIB, [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
    if binding:
        try:
            obj, torch_lib = made.result()
            tmp = BINDING + ".tmp"
            # torch's libraries are in the process when the binding is imported
            link("the binding", tmp, BINDING,
                 ["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-l:liblynx.so", "-Wl,-rpath,$ORIGIN", "-L", torch_lib,
                  "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
            with open(BINDING + ".of", "w") as f:
                f.write(_binding_of())
        except (RuntimeError, ImportError, OSError) as e:
            if os.path.exists(BINDING):
                os.remove(BINDING)   # built from other sources, or for another torch
            warnings.warn(f"{os.path.basename(BINDING)} was not built, the serving-step calls of the Python package "
                          f"need it: {e}")
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
