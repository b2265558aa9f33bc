"""Build libpq.so in-tree with nvcc for sm_100a.

    python -m rotation_int4_w4a4_b200.build [--force] [--verbose]

Objects go to ``_build/`` at the repository root; the shared library to
``rotation_int4_w4a4_b200/_lib/libpq.so``.  The CUDA runtime is linked statically, so the
library depends only on the driver (``libcuda``) at run time.  Beside it lies ``_pqcall-<torch><Python>.so``,
the Python module through which pq.py makes its quickest calls, compiled against the installed torch, whose
version its name holds; where that fails the library is built all the same.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libpq.so")
OBJDIR = os.path.join(ROOT, "_build")
SOURCES = ["pq_host.cpp", "transform.cu", "smooth_rows.cu", "rotate_mma.cu", "gemm.cu", "gemm_small.cu", "gemv.cu", "rrs.cu", "rows_small.cu", "gemm_static_scratch.cu",
           "ops_host.cpp", "quant8.cu", "w8a8.cu", "quant_fp4.cu", "fp4.cu", "kv4_append.cu", "kv4_attention.cu", "kv4_prompt.cu"]
HEADERS = ["internal.h", "ptx.cuh", "rows.cuh", "nan_max.cuh", "kv4.h", "kv4_device.cuh", "quant_fp4.cuh", "ptx_fp4.cuh"]
CALL_SOURCE = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC,-O2,-Wall",
                     "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_folder() -> str | None:
    """Where torch lies (found, not imported), None without it."""
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec and spec.submodule_search_locations else None


def torch_version() -> str:
    """The installed torch's version, "none" without one."""
    try:
        with open(os.path.join(_torch_folder() or "", "version.py")) as f:
            found = re.search(r"^__version__\s*=\s*['\"]([^'\"]+)", f.read(), re.M)
    except OSError:
        found = None
    return found.group(1) if found else "none"


def call_lib_name(version: str) -> str:
    """The compiled module's file for this Python and a torch of that version, whose objects it reads in place."""
    return "_pqcall-" + re.sub(r"[^\w.+]", "_", version) + (sysconfig.get_config_var("EXT_SUFFIX") or ".so")


CALL_LIB = os.path.join(LIBDIR, call_lib_name(torch_version()))


def _call_command(source: str | None = None, target: str | None = None) -> list[str] | None:
    """The compiler's command for the module, None without torch: the library needs none."""
    torch = _torch_folder()
    if torch is None:
        return None
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.isabs(nvcc()) else "/usr/local/cuda"
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return ([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall"] + ["-isystem" + d for d in include] +
            [source or CALL_SOURCE, "-o", target or CALL_LIB, "-L" + os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])


def _run(cmd: list[str], verbose: bool) -> subprocess.CompletedProcess:
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:                                 # no such compiler
        res = subprocess.CompletedProcess(cmd, 127, "", f"{e}\n")
    if verbose or res.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + res.stdout + res.stderr)
    return res


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "pq.h")]
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJDIR, src + ".o")
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            extra = ["-Xptxas", "-v"] if verbose and src.endswith(".cu") else []
            jobs.append([nvcc()] + NVCC_FLAGS + extra + ["-c", s, "-o", o])
    for other in glob.glob(os.path.join(glob.escape(LIBDIR), "_pqcall*.so")):   # of another torch, and of other sources
        if other != CALL_LIB and _stale(other, [CALL_SOURCE, hdrs[-1]]):
            os.remove(other)
    stale = force or _stale(CALL_LIB, [CALL_SOURCE, hdrs[-1]])
    call = _call_command() if stale else None
    if stale and call is None:
        sys.stderr.write("torch is not installed: the module _pqcall, which reads its tensors, is left out\n")
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        made = ex.submit(_run, call, verbose) if call else None
        for cmd, res in zip(jobs, ex.map(lambda c: _run(c, verbose), jobs)):
            if res.returncode != 0:
                raise RuntimeError(f"compilation failed: {' '.join(cmd)}")
    if force or jobs or _stale(LIB, objs):
        cmd = [nvcc()] + ARCH + ["-shared", "-o", LIB] + objs + ["-cudart", "static"]
        if _run(cmd, verbose).returncode != 0:
            raise RuntimeError("link of libpq.so failed")
    # The module only makes calls quicker: the library does without it.  One of other sources goes: it might call by other signatures.
    if stale and (made is None or made.result().returncode != 0):
        if os.path.exists(CALL_LIB):
            os.remove(CALL_LIB)
        if made:
            sys.stderr.write("the module _pqcall could not be compiled (above): calls go through ctypes, some 5 us slower\n")
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(a.force, a.verbose))
