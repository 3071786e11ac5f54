"""Builds ``libnt.so`` (the C ABI library of include/nt.h) in-tree with nvcc for sm_103a, and
``_ntbind.so``, the native part of its Python binding, with g++.

Each ``csrc/*.cu`` translation unit is compiled in its own nvcc process (in parallel), then
linked into ``packed_weight_gemv_gb300/_lib/libnt.so``. Re-running is incremental: a unit is
rebuilt when it or any header is newer than its object.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libnt.so")
BIND = os.path.join(OUT_DIR, "_ntbind.so")
BIND_STAMP = BIND + ".for"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libnt")
    return path


def _flags(extra=()):
    return [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
            "-I", CSRC, "--expt-relaxed-constexpr", *extra]


def binding_stamp() -> str:
    """What the native binding is compiled against besides its sources."""
    return "\n".join((sys.version, sysconfig.get_paths()["include"], importlib.metadata.version("torch"),
                      importlib.util.find_spec("torch").origin))


def binding_is_current() -> bool:
    src = os.path.join(CSRC, "nt_binding.cpp")
    newest = max(os.path.getmtime(f) for f in (src, os.path.join(INCLUDE, "nt.h")))
    if not os.path.exists(BIND) or os.path.getmtime(BIND) < newest or not os.path.exists(BIND_STAMP):
        return False
    with open(BIND_STAMP) as f:
        return f.read() == binding_stamp()


def build_binding() -> str:
    """csrc/nt_binding.cpp against this machine's torch and Python headers; again when either is another one."""
    if binding_is_current():
        return BIND
    src = os.path.join(CSRC, "nt_binding.cpp")
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = BIND + f".{os.getpid()}.tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(torch_dir, "include"), "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", INCLUDE, src, "-o", tmp, "-L", os.path.join(torch_dir, "lib"),
           "-Wl,-rpath," + os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on nt_binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)
    with open(BIND_STAMP, "w") as f:
        f.write(binding_stamp())
    return BIND


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    newest_header = max((os.path.getmtime(h) for h in headers), default=0.0)
    tool = nvcc()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        if (not ptxas_info and os.path.exists(obj)
                and os.path.getmtime(obj) >= max(os.path.getmtime(src), newest_header)):
            return obj, ""
        cmd = [tool, *_flags(["-Xptxas", "-v"] if ptxas_info else []), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        binding = ex.submit(build_binding)
        results = list(ex.map(compile_one, sources))
        binding.result()
    objs = [o for o, _ in results]
    if verbose or ptxas_info:
        for _, log in results:
            if log:
                sys.stderr.write(log)
    if (not os.path.exists(LIB)
            or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs)):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [tool, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="--ptxas" in sys.argv))
