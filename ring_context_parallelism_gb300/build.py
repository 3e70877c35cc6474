"""Build in-tree: every .cu under csrc/ compiled for sm_103a in parallel and
linked into libra.so, which exports the C ABI of include/ra.h; and _paged.so,
the CPython extension that binds the calls over paged sequences, linked against
libra.so and PyTorch."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libra.so")
PAGED = os.path.join(HERE, "_paged.so")
PAGED_SRC = os.path.join(CSRC, "paged_binding.cpp")
ROOT = os.path.dirname(HERE)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libra.so")
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return hs + [os.path.join(ROOT, "include", "ra.h")]


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _paged_made_for() -> str:
    """What the binding's compiled form depends on besides its source."""
    import torch
    return f"torch {torch.__version__} at {_torch_dir()}, python {sys.version}"


def _paged_compile(obj):
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-isystem", inc, "-isystem", cuda,
            "-isystem", sysconfig.get_paths()["include"], "-I", os.path.join(ROOT, "include"), "-c", PAGED_SRC, "-o", obj]


def _paged_link(obj, target):
    lib = os.path.join(_torch_dir(), "lib")
    return ["g++", "-shared", "-o", target, obj, "-L", HERE, "-l:libra.so", "-L", lib, "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hs = headers()
    srcs = sources()
    objs = []
    jobs = []
    # the binding first: with PyTorch's headers it is among the longer compilations
    paged_obj = os.path.join(BUILD, "paged_binding.o")
    stamp = os.path.join(BUILD, "paged_binding.txt")
    made_for = _paged_made_for()
    paged_stale = (force or _stale(paged_obj, [PAGED_SRC, os.path.join(ROOT, "include", "ra.h")]) or
                   not os.path.exists(stamp) or open(stamp).read() != made_for)
    if paged_stale:
        jobs.append(_paged_compile(paged_obj))
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + hs):
            cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
            jobs.append(cmd)
    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            for cmd, r in ex.map(run, jobs):
                if verbose or r.returncode:
                    sys.stderr.write(r.stdout + r.stderr)
                if r.returncode:
                    raise RuntimeError(f"compilation failed: {' '.join(cmd)}")

    def link(target, cmd):
        tmp = target + f".tmp{os.getpid()}"
        r = subprocess.run(cmd(tmp), capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError(f"link of {os.path.basename(target)} failed")
        os.replace(tmp, target)
    if force or jobs or _stale(LIB, objs):
        link(LIB, lambda tmp: [nvcc(), *ARCH, "-shared", "-o", tmp, *objs])
    if paged_stale or _stale(PAGED, [paged_obj]):
        link(PAGED, lambda tmp: _paged_link(paged_obj, tmp))
        with open(stamp, "w") as f:
            f.write(made_for)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
