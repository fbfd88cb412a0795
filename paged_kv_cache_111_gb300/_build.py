"""Build libpagedkv.so in-tree with nvcc for sm_103a (no CMake, no torch extension).

Each .cu file under csrc/ is compiled in parallel to an object file, then all
are linked into one shared library beside this file.  The Python module that
marshals the int8 calls (csrc/py_calls.c, no torch headers) is compiled with
the host's C compiler and linked to it; its name carries the interpreter's tag,
since it holds that one's object layout.  Without Python's headers it is left
out: the int8 calls then refuse, all others work.  The build is skipped when
what it makes is newer than every source and header.
"""

from __future__ import annotations

import concurrent.futures
import glob
import os
import shlex
import shutil
import subprocess
import sys
import sysconfig
from typing import List, Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libpagedkv.so")
CALLS = os.path.join(PKG, "_py_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
OBJDIR = os.path.join(PKG, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libpagedkv.so")


def sources() -> List[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> List[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(CSRC, "*.c")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def python_headers() -> Optional[str]:
    """The running interpreter's header folder, None where it is not installed."""
    folder = sysconfig.get_paths()["include"]
    return folder if os.path.exists(os.path.join(folder, "Python.h")) else None


def up_to_date() -> bool:
    made = [LIB] + ([CALLS] if python_headers() else [])
    if not all(os.path.exists(f) for f in made):
        return False
    t = min(os.path.getmtime(f) for f in made)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build_calls(out: str = CALLS) -> None:
    """Compile csrc/py_calls.c for the running interpreter."""
    headers = python_headers()
    if headers is None:
        print(f"no Python.h for {sys.executable}: built without the int8 calls from Python", file=sys.stderr)
        return
    cc = shlex.split(os.environ.get("CC", "")) or [shutil.which("gcc") or "cc"]
    tmp = out + f".tmp{os.getpid()}"
    res = subprocess.run([*cc, "-O2", "-std=c11", "-Wall", "-fPIC", "-shared", "-I", INCLUDE, "-I", headers,
                          os.path.join(CSRC, "py_calls.c"), "-o", tmp, "-L", PKG, "-l:" + os.path.basename(LIB),
                          "-Wl,-rpath,$ORIGIN"], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"compiling py_calls.c failed:\n{res.stderr}")
    os.replace(tmp, out)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{res.stderr}")
        if verbose and res.stderr:
            print(res.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    res = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking libpagedkv.so failed:\n{res.stderr}")
    os.replace(tmp, LIB)
    build_calls()
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
