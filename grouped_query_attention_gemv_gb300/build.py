"""Build libgqa.so in-tree: one nvcc per CUDA translation unit (in parallel),
then a shared-library link; and beside it the Python extension gqa_binding.so
(host code only), linked to it. Target: GB300, sm_103a only.

    python -m grouped_query_attention_gemv_gb300.build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import fcntl
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "lib")
OBJ_DIR = os.path.join(OUT_DIR, "obj")
LIB = os.path.join(OUT_DIR, "libgqa.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(OUT_DIR, "gqa_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libgqa")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _torch_dir(sub: str) -> str:
    import torch
    return os.path.join(os.path.dirname(torch.__file__), sub)


def _binding_cmd(obj: str):
    import torch
    inc = _torch_dir("include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", inc, "-I", cuda, "-c", BINDING_SRC, "-o", obj]


def _deps():
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    hdrs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hdrs + [os.path.abspath(__file__)]


def _stale(target: str, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(i) > t for i in inputs)


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = True) -> str:
    """Compile and link; return the path of libgqa.so. Raises on failure. One
    build at a time works on the tree: another waits for it, and finds its files."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    with open(os.path.join(OUT_DIR, ".lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        return _build(force, verbose_ptxas, quiet)


def _build(force: bool, verbose_ptxas: bool, quiet: bool) -> str:
    cc = nvcc()
    deps = _deps()
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or verbose_ptxas or _stale(obj, [src] + deps):
            cmd = [cc, *ARCH, *FLAGS, "-c", src, "-o", obj]
            if verbose_ptxas:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    bobj = os.path.join(OBJ_DIR, "binding.o")
    rebind = force or _stale(bobj, [BINDING_SRC, os.path.join(INCLUDE, "gqa.h"), os.path.abspath(__file__)])
    if rebind:
        jobs.insert(0, _binding_cmd(bobj))

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for cmd, r in ex.map(run, jobs):
            if r.returncode != 0:
                raise RuntimeError(f"{os.path.basename(cmd[0])} failed for {cmd[-3]}:\n{r.stdout}\n{r.stderr}")
            if verbose_ptxas or not quiet:
                sys.stderr.write(r.stderr)
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if rebind or _stale(BINDING, [bobj]):
        tmp = BINDING + ".tmp"
        r = subprocess.run(["g++", "-shared", "-o", tmp, bobj, "-L", OUT_DIR, "-l:libgqa.so", "-Wl,-rpath,$ORIGIN",
                            "-L", _torch_dir("lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas, quiet=False))
