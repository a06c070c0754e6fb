"""Builds the shared library ``_build/libmuon_gb300.so`` in-tree with nvcc
for sm_103a only, and ``_build/_torch_calls.<versions>.so``, the Python module
that does the torch layer's checks and calls.  Translation units compile in
parallel; no cmake.

    python -m muon_newton_schulz_gb300.build [--force] [-v] [-DNAME=VALUE ...] [--out DIR]

``-D`` options are passed to every translation unit (for example the
pipeline shape macros of k_tc.cu); with ``--out`` the objects and the
library go to another directory instead of ``_build``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB_NAME = "libmuon_gb300.so"
LIB = os.path.join(BUILD, LIB_NAME)
INCLUDE = os.path.join(ROOT, "include")
# One built for another Python or torch has undefined calls: each has its name.
CALLS_STEM = f"_torch_calls.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}"
CALLS_NAME = CALLS_STEM + ".so"
CALLS = os.path.join(BUILD, CALLS_NAME)

CUDA_SOURCES = ["k_elementwise.cu", "k_simt_f32.cu", "k_tc.cu", "muon_noalloc.cu", "k_adamw.cu", "k_moe.cu", "k_embed.cu",
                "k_saved8.cu", "k_ffn.cu", "k_ffn_tc.cu",
                "k_ffn_few.cu", "k_ffn_lines.cu"]
CXX_SOURCES = ["muon_api.cpp", "train_api.cpp", "layer_api.cpp", "ffn_api.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _cuda_home() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if home and os.path.isdir(home):
        return home
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    return r.returncode, " ".join(cmd), r.stdout


def _stale(obj: str, deps) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, defines=None, out: str | None = None) -> str:
    """Compiles what changed and links the library; returns its path."""
    cuda = _cuda_home()
    nvcc = os.path.join(cuda, "bin", "nvcc")
    bdir = out or BUILD
    lib = os.path.join(bdir, LIB_NAME)
    os.makedirs(bdir, exist_ok=True)
    defs = [f"-D{d}" for d in (defines or [])]
    if defs:
        force = True
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(INCLUDE, "muon.h"))
    common = ["-O3", "-std=c++17", "-I", INCLUDE, "-I", CSRC, "-I", os.path.join(cuda, "include"), *defs]
    jobs = []
    objs = []
    for src in CUDA_SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(bdir, src + ".o")
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc, *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", *common, "-c", s, "-o", o])
    for src in CXX_SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(bdir, src + ".o")
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc, "-x", "c++", "-Xcompiler", "-fPIC", *common, "-c", s, "-o", o])
    # the torch layer's module: needs torch's headers, not nvcc
    torch_dir = os.path.dirname(torch.__file__)
    calls_src, calls_obj = os.path.join(CSRC, "torch_calls.cpp"), os.path.join(bdir, CALLS_STEM + ".o")
    calls_lib = os.path.join(bdir, CALLS_NAME)
    compile_calls = force or _stale(calls_obj, [calls_src, headers[-1]])
    if compile_calls:
        inc = os.path.join(torch_dir, "include")
        jobs.append(["g++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
                     "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
                     "-c", calls_src, "-o", calls_obj])
    if jobs:
        with ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
            results = list(ex.map(_run, jobs))
        for rc, cmd, text in results:
            if verbose or rc != 0:
                sys.stderr.write(cmd + "\n" + text)
            if rc != 0:
                raise RuntimeError("compilation failed: " + cmd + "\n" + text)
    if compile_calls or _stale(calls_lib, [calls_obj]):
        tdir = os.path.join(torch_dir, "lib")
        tmp = calls_lib + ".tmp"
        rc, cmd, text = _run(["g++", "-shared", "-o", tmp, calls_obj, "-L" + tdir, "-ltorch_python", "-ltorch_cpu",
                              "-lc10", "-Wl,-rpath," + tdir])
        if rc != 0:
            raise RuntimeError("link failed: " + cmd + "\n" + text)
        os.replace(tmp, calls_lib)
    if force or jobs or _stale(lib, objs):
        tmp = lib + ".tmp"
        rc, cmd, text = _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lrt", "-lpthread"])
        if rc != 0:
            raise RuntimeError("link failed: " + cmd + "\n" + text)
        os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    args = sys.argv[1:]
    defines = [a[2:] for a in args if a.startswith("-D")]
    out = args[args.index("--out") + 1] if "--out" in args else None
    print(build(force="--force" in args, verbose="-v" in args, defines=defines, out=out))
