"""Build the CUDA library libkda_prefill.so (nvcc, sm_100a only) and the Python binding of its
layer operators, _layer_bind.so (g++, against torch), in-tree.  The library needs nvcc alone; the
binding is left out, with a note, where torch, g++ or Python's headers are missing.

Usage: python -m kda_chunked_recurrent_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libkda_prefill.so")
SOURCES = ["kda_api.cu", "kda_schedule.cu", "kda_prepare.cu", "kda_recurrence.cu",
           "kda_fused.cu", "kda_stream.cu", "kda_token.cu", "kda_noalloc.cu",
           "kda_layer_api.cu", "kda_conv.cu", "kda_scan.cu", "kda_norm.cu"]
HEADERS = ["kda_common.cuh", "sm100_primitives.cuh", "kda_prepare.cuh", "kda_recurrence.cuh",
           "kda_chain.cuh", "kda_token.cuh", "kda_layer.cuh"]
PUBLIC = ["kda_prefill.h", "kda_layer.h"]
BIND = os.path.join(PKG, "_layer_bind.so")
BIND_SOURCE = "kda_layer_bind.cpp"


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files += [os.path.join(ROOT, "include", f) for f in PUBLIC]
    return files


def _bind_inputs():
    return [os.path.join(CSRC, BIND_SOURCE)] + [os.path.join(ROOT, "include", f) for f in PUBLIC]


def _stale(target: str, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in inputs)


def _missing_for_bind() -> list:
    """What the binding's build needs and this machine lacks."""
    header = os.path.join(sysconfig.get_paths()["include"], "Python.h")
    return [what for what, found in (("torch", importlib.util.find_spec("torch")),
                                     ("g++", shutil.which("g++")),
                                     ("Python.h", os.path.exists(header))) if not found]


def needs_build() -> bool:
    return _stale(LIB, _inputs()) or (_stale(BIND, _bind_inputs()) and not _missing_for_bind())


def _bind_command(out: str) -> list:
    """g++ for the binding: torch's headers and libraries, the library beside it."""
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api",
                                                        "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"],
           os.path.join(ROOT, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in inc:
        cmd += ["-isystem", d]
    return cmd + [os.path.join(CSRC, BIND_SOURCE), "-o", out, "-L", os.path.join(base, "lib"),
                  "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
                  "-L", PKG, "-l:libkda_prefill.so", "-Wl,-rpath,$ORIGIN"]


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _stale(LIB, _inputs()):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo",
               "-std=c++17", "--threads", "0", "-Xcompiler", "-fPIC", "-shared",
               "-Xlinker", "-soname=libkda_prefill.so", "-I", os.path.join(ROOT, "include"),
               "-o", tmp] + [os.path.join(CSRC, f) for f in SOURCES]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    missing = _missing_for_bind()
    if missing:
        print(f"{os.path.basename(BIND)} not built (the Python functions of the layer operators "
              f"need it), missing: {', '.join(missing)}", file=sys.stderr, flush=True)
    elif force or _stale(BIND, _bind_inputs()):
        tmp = BIND + f".tmp{os.getpid()}"
        cmd = _bind_command(tmp)
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, BIND)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
    sys.exit(0)
