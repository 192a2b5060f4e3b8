"""Build the CUDA library ``libmono.so`` in-tree with nvcc for sm_100a, and the Python module ``_tensor_args``.

    python -m learned_product_hash_proj_b200.build [--force] [-j N]

Each ``csrc/*.cu`` is compiled to ``_build/<name>.o`` (parallel), then linked
into ``learned_product_hash_proj_b200/libmono.so``.  ptxas register and
shared-memory reports go to ``_build/<name>.ptxas.txt``.  ``csrc/tensor_args.cc``
is host code for the running Python and torch (g++, with torch's DLPack header).
The package works without it: where it does not compile, a warning says so.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmono.so")
ARGS_SRC = os.path.join(CSRC, "tensor_args.cc")
# the suffix names the Python that it is built for, so that no other one loads it
ARGS_LIB = os.path.join(PKG, "_tensor_args" + sysconfig.get_config_var("EXT_SUFFIX"))
ARGS_KEY = os.path.join(BUILD, "tensor_args.key")  # what the last build of it, successful or not, was for

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libmono.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(i) > t for i in inputs)


def _compile(src: str) -> str:
    name = os.path.splitext(os.path.basename(src))[0]
    obj = os.path.join(BUILD, name + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(BUILD, name + ".ptxas.txt"), "w") as f:
        f.write(res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr[-6000:]}")
    return obj


def _args_key() -> str:
    return f"{os.path.basename(ARGS_LIB)} torch {importlib.metadata.version('torch')}"


def _args_stale() -> bool:
    inputs = [ARGS_SRC, os.path.join(INCLUDE, "mono.h")]
    if _stale(ARGS_KEY, inputs):
        return True
    with open(ARGS_KEY) as f:
        last, built = f.read().rsplit("\n", 1)
    return last != _args_key() or (built == "built" and _stale(ARGS_LIB, inputs))


def _build_tensor_args() -> bool:
    """Compile the module; where that fails, leave none behind and warn."""
    try:
        torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
        tmp = ARGS_LIB + ".tmp"
        cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-fvisibility=hidden",
               "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch_dir, "include"), "-I", INCLUDE,
               ARGS_SRC, "-o", tmp]
        res = subprocess.run(cmd, capture_output=True, text=True)
        why = (res.stderr[-4000:] or f"g++ ended with {res.returncode}") if res.returncode else ""
    except OSError as e:
        why = str(e)
    if why:
        warnings.warn(f"{os.path.basename(ARGS_LIB)} was not built: the dense operators check their tensors in Python\n"
                      + why, stacklevel=2)
        if os.path.exists(ARGS_LIB):
            os.remove(ARGS_LIB)
    else:
        os.replace(tmp, ARGS_LIB)
    with open(ARGS_KEY, "w") as f:
        f.write(_args_key() + ("\nfailed" if why else "\nbuilt"))
    return not why


def build(force: bool = False, jobs: int | None = None, verbose: bool = False) -> str:
    """Compile (if stale) and link libmono.so, and, where it compiles, the module beside it; returns libmono.so's path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    deps = _deps()
    todo = [s for s in srcs if force or _stale(os.path.join(BUILD, os.path.splitext(os.path.basename(s))[0] + ".o"),
                                               [s, *deps])]
    jobs = jobs or min(len(todo) or 1, os.cpu_count() or 4)
    if todo:
        with cf.ThreadPoolExecutor(jobs) as ex:
            for obj in ex.map(_compile, todo):
                if verbose:
                    print("compiled", obj, file=sys.stderr)
    objs = [os.path.join(BUILD, os.path.splitext(os.path.basename(s))[0] + ".o") for s in srcs]
    if force or todo or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stderr[-4000:]}")
        os.replace(tmp, LIB)
    untagged = os.path.join(PKG, "_tensor_args.so")  # of earlier builds: any Python would load it
    if os.path.exists(untagged):
        os.remove(untagged)
    if (force or _args_stale()) and _build_tensor_args() and verbose:
        print("compiled", ARGS_SRC, file=sys.stderr)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-j", type=int, default=None)
    a = ap.parse_args()
    print(build(force=a.force, jobs=a.j, verbose=True))
