"""Compile the CUDA sources into ``libmoba_gb300.so`` (sm_103a only), and the
binding of the calls whose host time counts into ``moba_calls.so``.

Each ``csrc/*.cu`` is compiled to an object in parallel, then nvcc links the
shared library in-tree next to this file; ``csrc/moba_calls.cpp`` (host code on torch's
headers, linked to that library) is compiled beside them.  Run ``python -m
long_context_sparse_moba_gb300.build`` or call :func:`build`.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoba_gb300.so")
CALLS = os.path.join(HERE, "moba_calls.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _calls_commands(lib: str):
    """The binding's object, its compile command, and the command that links it to ``to``."""
    root = os.path.dirname(torch.__file__)
    libs = os.path.join(root, "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    obj = os.path.join(BUILD, f"moba_calls-{torch.__version__}.o")  # (of one version of torch)
    cxx = os.environ.get("CXX") or "g++"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE,
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                "-isystem", os.path.join(root, "include"),
                "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
                "-c", os.path.join(CSRC, "moba_calls.cpp"), "-o", obj]
    link = lambda to: [cxx, "-shared", "-o", to, obj, "-L", os.path.dirname(lib), "-l:" + os.path.basename(lib),
                       "-Wl,-rpath,$ORIGIN", "-L", libs, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda",
                       "-ltorch", "-lc10_cuda", "-lc10"]
    return obj, compile_, link


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    objs, jobs = [], []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
            if verbose:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    calls_obj, calls_compile, calls_link = _calls_commands(LIB)
    if force or _stale(calls_obj, [os.path.join(CSRC, "moba_calls.cpp"), os.path.join(INCLUDE, "moba.h")]):
        jobs.insert(0, calls_compile)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("compiling failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        return r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for out in ex.map(run, jobs):
            if verbose and out:
                print(out, file=sys.stderr)
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    stamp = os.path.join(BUILD, "moba_calls.torch")  # the version that CALLS is linked to
    linked = ""
    if os.path.exists(stamp):
        with open(stamp) as f:
            linked = f.read()
    if force or jobs or _stale(CALLS, [calls_obj]) or linked != torch.__version__:
        tmp = CALLS + f".tmp{os.getpid()}"
        run(calls_link(tmp))
        os.replace(tmp, CALLS)
        with open(stamp + f".tmp{os.getpid()}", "w") as f:
            f.write(torch.__version__)
        os.replace(f.name, stamp)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
