"""Build libhga.so (sm_100a) in-tree with nvcc, and its Python binding with g++.

Each CUDA source under csrc/ is compiled to an object in _build/ (in
parallel), then linked into long_context_rope_b200/libhga.so; csrc/py_bind.cpp
becomes long_context_rope_b200/_hga_bind.so, which links to it. The binding reads
torch's own objects, so another version of torch or Python builds it again. Run as
``python -m long_context_rope_b200.build`` or call ``build()``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libhga.so")
BIND = os.path.join(PKG, "_hga_bind.so")
BIND_SRC = os.path.join(CSRC, "py_bind.cpp")
BIND_FOR = os.path.join(OUT_DIR, "_hga_bind.for")  # what BIND was built for

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-O2", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    """Compile every CUDA source for sm_100a, link libhga.so and build its Python
    binding. Returns the library's path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs, hdrs = _sources(), _headers()
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(OUT_DIR, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            cmd = [nvcc(), *ARCH, *FLAGS, "-c", s, "-o", o]
            if ptxas_v:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        for cmd, r in zip(jobs, results):
            if verbose or r.returncode != 0 or ptxas_v:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed for {cmd[-3]}")
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            raise RuntimeError("link of libhga.so failed")
        os.replace(tmp, LIB)
    if force or _bind_stale():
        _build_bind()
    return LIB


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def built_for() -> str:
    """The versions whose objects the binding reads: torch's and Python's."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        version = re.search(r"^__version__ = ['\"](.+)['\"]", f.read(), re.M).group(1)
    return f"torch {version}, {sysconfig.get_config_var('SOABI')}"


def _bind_stale() -> bool:
    if _stale(BIND, [BIND_SRC, os.path.join(INCLUDE, "hga.h")]) or not os.path.exists(BIND_FOR):
        return True
    with open(BIND_FOR) as f:
        return f.read() != built_for()


def _build_bind() -> None:
    torch_dir = _torch_dir()
    tmp = BIND + f".tmp{os.getpid()}"
    inc = os.path.join(torch_dir, "include")
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f'-DHGA_BUILT_FOR="{built_for()}"', f"-I{INCLUDE}", f"-I{sysconfig.get_paths()['include']}", f"-isystem{inc}",
           "-isystem" + os.path.join(inc, "torch", "csrc", "api", "include"), BIND_SRC, "-o", tmp,
           f"-L{PKG}", "-l:libhga.so", "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("build of _hga_bind.so failed")
    os.replace(tmp, BIND)
    with open(BIND_FOR, "w") as f:
        f.write(built_for())


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_v="--ptxas-v" in sys.argv)
    print(LIB)
