"""Builds libcsa.so (the CUDA kernels + C ABI) in-tree for sm_100a with nvcc.

Each .cu file under csrc/ compiles to an object in parallel; the objects link into
long_context_compressed_04_b200/libcsa.so with the CUDA runtime linked statically, so the
library needs no CUDA shared library besides the driver at run time.  csrc/marshal.cpp, the
Python binding's compiled argument marshalling, builds beside it with the host compiler
against the installed torch (_csa_marshal.so); where that fails, the binding does without.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libcsa.so")
MARSHAL = os.path.join(HERE, "_csa_marshal.so")
OBJ_DIR = os.path.join(HERE, "_build")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libcsa")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build_marshal(force: bool = False) -> str:
    import sysconfig

    import torch
    src = os.path.join(CSRC, "marshal.cpp")
    troot = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "g++", "-O2", "-shared", "-fPIC",
           "-std=c++17", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DCSA_TORCH="{torch.__version__}"', f'-DCSA_PYTHON="{sys.implementation.cache_tag}"',
           "-I" + sysconfig.get_paths()["include"], "-isystem", os.path.join(troot, "include"),
           "-isystem", os.path.join(troot, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), src,
           "-L" + os.path.join(troot, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    # torch's headers are not among the files looked at: the command, which names their version,
    # is kept beside the objects, and another one builds again
    stamp = os.path.join(OBJ_DIR, "marshal.cmd")
    same = os.path.exists(stamp) and open(stamp).read() == "\n".join(cmd)
    if same and not force and not _stale(MARSHAL, [src, os.path.join(ROOT, "include", "csa.h")]):
        return MARSHAL
    r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("build of _csa_marshal.so failed")
    os.replace(tmp, MARSHAL)
    os.makedirs(OBJ_DIR, exist_ok=True)
    with open(stamp, "w") as f:
        f.write("\n".join(cmd))
    return MARSHAL


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    srcs = _sources()
    hdrs = _headers()
    os.makedirs(OBJ_DIR, exist_ok=True)
    cc = nvcc()
    marshal = concurrent.futures.ThreadPoolExecutor(max_workers=1).submit(build_marshal, force)
    jobs = []
    for s in srcs:
        obj = os.path.join(OBJ_DIR, os.path.basename(s)[:-3] + ".o")
        if force or _stale(obj, [s] + hdrs):
            cmd = [cc, *ARCH, *FLAGS, "-c", s, "-o", obj]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)
    if jobs:
        with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        failed = [r for r in results if r.returncode != 0]
        for r in results:
            if verbose or r.returncode != 0 or ptxas_info:
                sys.stderr.write(r.stdout + r.stderr)
        if failed:
            raise RuntimeError(f"nvcc failed on {len(failed)} file(s)")
    objs = [os.path.join(OBJ_DIR, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if force or jobs or _stale(OUT, objs):
        tmp = OUT + f".tmp{os.getpid()}"
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link of libcsa.so failed")
        os.replace(tmp, OUT)
    try:
        marshal.result()
    except Exception as e:      # noqa: BLE001  (no torch, no Python headers, no host compiler)
        # the library stands without it and the binding does the same in Python, more slowly; one of
        # an older source must not stay
        if os.path.exists(MARSHAL):
            os.remove(MARSHAL)
        sys.stderr.write(f"_csa_marshal.so was not built ({type(e).__name__}: {e}): the binding goes on without it\n")
    return OUT


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(OUT)
