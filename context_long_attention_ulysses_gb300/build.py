"""Build libusp.so (the C-ABI library) in-tree for sm_103a with nvcc.

Each CUDA translation unit compiles in parallel; the objects link into
``_build/libusp.so`` against the shared CUDA runtime, and ``binding.cpp``, the
Python side of a decoding step's calls, into ``_build/uspbinding.<Python's ABI>.so``.  The
library needs nothing of Python: it is linked whatever becomes of the binding,
which is left out, with a note, where Python's C headers are missing.  Run as
``python -m context_long_attention_ulysses_gb300.build``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libusp.so")
BINDING = os.path.join(BUILD, "uspbinding" + sysconfig.get_config_var("EXT_SUFFIX"))  # (of this Python alone)
SOURCES = ["api.cu", "remap.cu", "attn_f32.cu", "attn_fwd.cu", "attn_bwd.cu", "ring.cu", "noalloc.cu", "diag.cu",
           "kv_append.cu", "rotary.cu", "pages.cu", "verify.cu", "paged_attn.cu", "paged_mma.cu", "paged_tc.cu", "paged_f32.cu"]
HEADERS = ["kernels.h", "ptx.cuh", "paged.cuh", "rotary.cuh", "cluster.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "-diag-suppress", "177"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libusp")


def _python_headers():
    """The directory of Python.h; None without it."""
    path = sysconfig.get_paths()["include"]
    return path if os.path.exists(os.path.join(path, "Python.h")) else None


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every translation unit for sm_103a and link libusp.so; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    header = os.path.join(os.path.dirname(HERE), "include", "usp.h")
    header_deps = [os.path.join(CSRC, h) for h in HEADERS] + [header]
    python = _python_headers()
    if python is None:
        print("Python.h not found: libusp.so is built without uspbinding.so, and the package's calls around the cache "
              "(usp_rotary_embed, usp_kv_append_axes, usp_pages_*, usp_verify_drafts) will raise", file=sys.stderr)
    binding = os.path.join(BUILD, os.path.splitext(os.path.basename(BINDING))[0] + ".o")
    objs = [os.path.join(BUILD, os.path.splitext(src)[0] + ".o") for src in SOURCES]
    units = [(src, o, header_deps, []) for src, o in zip(SOURCES, objs)]
    if python is not None:
        units.append(("binding.cpp", binding, [header], ["-I", python]))
    procs = []
    for src, o, deps, flags in units:
        s = os.path.join(CSRC, src)
        if force or _stale(o, [s, *deps]):
            cmd = [nvcc, *flags, *ARCH, *FLAGS, "-c", s, "-o", o + ".tmp"]
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append((subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT), o, cmd))
    failed = {}
    for p, o, cmd in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed[o] = " ".join(cmd) + "\n" + out.decode(errors="replace")
        else:
            os.replace(o + ".tmp", o)
            if verbose and out:
                print(out.decode(errors="replace"))
    links = [(LIB, objs, [])]
    if python is not None:
        links.append((BINDING, [binding], ["-L", os.path.dirname(LIB), "-lusp", "-Xlinker", "-rpath=$ORIGIN"]))
    for target, parts, libs in links:
        if not failed.keys() & set(parts) and (force or _stale(target, parts)):
            tmp = target + f".tmp{os.getpid()}"
            cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *parts, *libs]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.check_call(cmd)
            os.replace(tmp, target)
        if failed.keys() & set(parts):
            raise RuntimeError("nvcc failed:\n" + "\n".join(failed.values()))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
